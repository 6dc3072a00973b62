"""Group norm with an activation, forward and backward.

PyTorch only supplies device memory and the stream; the arithmetic runs in
libdeft.so (``deft_norm_forward``, ``deft_norm_backward``) through the binding
in ``_lib``.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import _lib
from ._stream import current_stream, elsewhere


class GroupNormAct:
    """y = act(gamma * (x - mean) * rstd + beta), the statistics over each of
    ``groups`` groups of consecutive channels of each image.

    ``layout``: "channels_first" (x is [n][c][s] in memory, such as the
    [n][c][h][w] that :class:`layer.DeformConv` writes, s = h * w) or
    "channels_last" ([n][s][c]).  ``act``: "none", "relu", "silu" or "gelu".
    ``dtype``: "bf16" or "f32", of x, gamma, beta, y and the gradients; the
    statistics are float32.  ``training``: hold the workspace that
    :meth:`backward` needs too.

    Calls run on the current stream of their device, whichever device is the
    current one; calls of one handle on several streams must be ordered by the
    caller, as they share the workspace (which the constructor zeroes on its
    current stream)."""

    def __init__(self, n, c, s, groups, eps=1e-5, act="none", layout="channels_first", dtype="bf16", training=False,
                 device="cuda"):
        for what, value, known in (("layout", layout, _lib.LAYOUTS), ("act", act, _lib.ACTIVATIONS),
                                   ("dtype", dtype, _DTYPES)):
            if value not in known:
                raise ValueError("%s must be one of %s, got %r" % (what, sorted(known), value))
        self.desc = _lib.deft_norm_desc(n, c, s, groups, _lib.LAYOUTS[layout], _lib.ACTIVATIONS[act],
                                        _lib.DEFT_BF16 if dtype == "bf16" else _lib.DEFT_F32, eps)
        self._index = torch.empty(0, device=device).get_device()
        with torch.cuda.device(self._index) if elsewhere(self._index) else contextlib.nullcontext():
            _lib.deft_norm_desc_validate(self.desc)
            self.ws_bytes = _lib.deft_norm_workspace_bytes(self.desc, 1 if training else 0)
        self.n, self.c, self.s, self.groups = n, c, s, groups
        self.tdtype, self.training = _DTYPES[dtype], training
        self.ws = torch.zeros(max(self.ws_bytes, 256), dtype=torch.uint8, device=device)
        self.device = self.ws.device
        self._stats = torch.empty((n, groups), dtype=torch.float32, device=device)
        # what each argument must be: elements and dtype
        self._image, self._channel, self._stat = (n * c * s, self.tdtype), (c, self.tdtype), (n * groups, torch.float32)
        self._kinds = dict(mean=self._stat, rstd=self._stat)
        self._kinds.update({k: self._image for k in ("x", "y", "dy", "dx")})
        self._kinds.update({k: self._channel for k in ("gamma", "beta", "dgamma", "dbeta")})

        # small calls wait for the host: the C functions are called without the binding's wrappers
        lib, self._ref, self._ws = _lib.load(), ctypes.byref(self.desc), self.ws.data_ptr()
        self._forward, self._backward = lib.deft_norm_forward, lib.deft_norm_backward

    def _unfit(self, t, kind):
        return (t.numel() != kind[0] or t.dtype is not kind[1] or t.get_device() != self._index
                or not t.is_contiguous())

    def _refuse(self, **tensors):
        for what, t in tensors.items():
            if t is not None and self._unfit(t, self._kinds[what]):
                raise ValueError("%s must be %d contiguous elements of %s on %s" % (
                    (what,) + self._kinds[what] + (self.device,)))

    def forward(self, x, gamma, beta, y=None, mean=None, rstd=None):
        """(y, mean, rstd); mean and rstd are float32 [n][groups], NaN where there are no positions."""
        unfit = self._unfit
        if unfit(x, self._image) or unfit(gamma, self._channel) or unfit(beta, self._channel):
            self._refuse(x=x, gamma=gamma, beta=beta)
        if y is not None or mean is not None or rstd is not None:
            self._refuse(y=y, mean=mean, rstd=rstd)
        if y is None:
            y = torch.empty_like(x)
        if mean is None:
            mean = torch.empty_like(self._stats)
        if rstd is None:
            rstd = torch.empty_like(self._stats)
        if self.s == 0:  # the C function writes nothing, then
            mean.fill_(math.nan)
            rstd.fill_(math.nan)
        if elsewhere(self._index):
            with torch.cuda.device(self._index):
                return self.forward(x, gamma, beta, y, mean, rstd)
        code = self._forward(self._ref, x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), y.data_ptr(), mean.data_ptr(),
                             rstd.data_ptr(), self._ws, self.ws_bytes, current_stream(self._index))
        if code:
            raise _lib.DeftError(code, "deft_norm_forward")
        return y, mean, rstd

    def backward(self, x, gamma, beta, mean, rstd, dy, out=None):
        """dict(dx, dgamma, dbeta).  ``out``: the buffers to write; what it
        leaves out or holds as None is not computed."""
        if not self.training:
            raise ValueError("backward needs training=True")
        unfit = self._unfit
        if (unfit(x, self._image) or unfit(gamma, self._channel) or unfit(beta, self._channel)
                or unfit(dy, self._image) or unfit(mean, self._stat) or unfit(rstd, self._stat)):
            self._refuse(x=x, gamma=gamma, beta=beta, mean=mean, rstd=rstd, dy=dy)
        if out is None:
            dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
            out = dict(dx=dx, dgamma=dgamma, dbeta=dbeta)
        else:
            if not out.keys() <= _GRADIENTS:
                raise ValueError("out may hold %s, got %s" % (sorted(_GRADIENTS), sorted(out)))
            dx, dgamma, dbeta = out.get("dx"), out.get("dgamma"), out.get("dbeta")
            if (dx is not None and unfit(dx, self._image) or dgamma is not None and unfit(dgamma, self._channel)
                    or dbeta is not None and unfit(dbeta, self._channel)):
                self._refuse(**out)
        if elsewhere(self._index):
            with torch.cuda.device(self._index):
                return self.backward(x, gamma, beta, mean, rstd, dy, out)
        code = self._backward(self._ref, x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), mean.data_ptr(),
                              rstd.data_ptr(), dy.data_ptr(), None if dx is None else dx.data_ptr(),
                              None if dgamma is None else dgamma.data_ptr(),
                              None if dbeta is None else dbeta.data_ptr(), self._ws, self.ws_bytes,
                              current_stream(self._index))
        if code:
            raise _lib.DeftError(code, "deft_norm_backward")
        return out


_GRADIENTS = {"dx", "dgamma", "dbeta"}
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
