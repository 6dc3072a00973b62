"""A device's current stream as the integer handle that the C ABI takes."""
from __future__ import annotations

import torch

# torch.cuda.current_stream() builds a Stream object for each call, a third of a
# small operator's time on the host; where torch has the plain getters, those are asked
_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def current_stream(index: int) -> int:
    """That of GPU `index`, a tensor's ``get_device()``."""
    if index < 0:
        raise ValueError("the tensors are not on a GPU")
    return _raw(index) if _raw is not None else torch.cuda.current_stream(index).cuda_stream


def elsewhere(index: int) -> bool:
    """Whether GPU `index` is not the current device.  The C ABI launches on the current one: every
    device's default stream has the handle 0."""
    return index >= 0 and _device() != index


class Lent:
    """Memory that a handle made for itself on one stream, used by calls on others.  Once the handle is gone torch
    gives such memory to the first stream's next allocations, but for streams that it was told of."""

    def __init__(self, index: int, tensors):
        self.index, self.tensors = index, list(tensors)
        self.streams = {current_stream(index) if index >= 0 else 0}

    def to(self, stream: int) -> int:
        """The stream, told of if it is new."""
        if stream not in self.streams:
            for t in self.tensors:
                t.record_stream(torch.cuda.current_stream(self.index))
            self.streams.add(stream)
        return stream
