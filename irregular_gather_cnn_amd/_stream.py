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
