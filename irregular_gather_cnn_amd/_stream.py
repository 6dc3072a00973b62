"""The device's current stream as the integer handle that the C ABI takes."""
from __future__ import annotations

import torch

# torch.cuda.current_stream() builds a Stream object for each call, a third of a
# small operator's time on the host; where torch has the plain getter, that is asked
_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def current_stream(device: torch.device) -> int:
    if _raw is not None and device.index is not None:
        return _raw(device.index)
    return torch.cuda.current_stream(device).cuda_stream
