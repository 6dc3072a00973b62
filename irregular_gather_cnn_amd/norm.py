"""Group norm with an activation, forward and backward.

PyTorch only supplies device memory and the stream; the arithmetic runs in
libdeft.so (``deft_norm_forward``, ``deft_norm_backward``) through the binding
in ``_lib``.
"""
from __future__ import annotations

import torch

from . import _lib


class GroupNormAct:
    """y = act(gamma * (x - mean) * rstd + beta), the statistics over each of
    ``groups`` groups of consecutive channels of each image.

    ``layout``: "channels_first" (x is [n][c][s] in memory, such as the
    [n][c][h][w] that :class:`layer.DeformConv` writes, s = h * w) or
    "channels_last" ([n][s][c]).  ``act``: "none", "relu", "silu" or "gelu".
    ``dtype``: "bf16" or "f32", of x, gamma, beta, y and the gradients; the
    statistics are float32.  ``training``: hold the workspace that
    :meth:`backward` needs too.

    Calls run on the device's current stream; calls of one handle on several
    streams must be ordered by the caller, as they share the workspace."""

    def __init__(self, n, c, s, groups, eps=1e-5, act="none", layout="channels_first", dtype="bf16", training=False,
                 device="cuda"):
        for what, value, known in (("layout", layout, _lib.LAYOUTS), ("act", act, _lib.ACTIVATIONS),
                                   ("dtype", dtype, _DTYPES)):
            if value not in known:
                raise ValueError("%s must be one of %s, got %r" % (what, sorted(known), value))
        self.desc = _lib.deft_norm_desc(n, c, s, groups, _lib.LAYOUTS[layout], _lib.ACTIVATIONS[act],
                                        _lib.DEFT_BF16 if dtype == "bf16" else _lib.DEFT_F32, eps)
        _lib.deft_norm_desc_validate(self.desc)
        self.n, self.c, self.s, self.groups = n, c, s, groups
        self.tdtype, self.device, self.training = _DTYPES[dtype], torch.device(device), training
        self.ws_bytes = max(_lib.deft_norm_workspace_bytes(self.desc, k) for k in range(2 if training else 1))
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=device)

    def _take(self, what, t, size, dtype):
        if t.numel() != size or t.dtype != dtype or t.device.type != self.device.type or not t.is_contiguous():
            raise ValueError("%s must be %d contiguous elements of %s on %s" % (what, size, dtype, self.device))

    def _take_inputs(self, x, gamma, beta):
        self._take("x", x, self.n * self.c * self.s, self.tdtype)
        self._take("gamma", gamma, self.c, self.tdtype)
        self._take("beta", beta, self.c, self.tdtype)

    def forward(self, x, gamma, beta, y=None, mean=None, rstd=None):
        """(y, mean, rstd); mean and rstd are float32 [n][groups]."""
        self._take_inputs(x, gamma, beta)
        stats = self.n * self.groups
        if y is None:
            y = torch.empty_like(x)
        else:
            self._take("y", y, x.numel(), self.tdtype)
        if mean is None:
            mean = torch.empty((self.n, self.groups), dtype=torch.float32, device=x.device)
        else:
            self._take("mean", mean, stats, torch.float32)
        if rstd is None:
            rstd = torch.empty((self.n, self.groups), dtype=torch.float32, device=x.device)
        else:
            self._take("rstd", rstd, stats, torch.float32)
        _lib.deft_norm_forward(self.desc, x, gamma, beta, y, mean, rstd, self.ws, self.ws_bytes,
                               torch.cuda.current_stream(x.device).cuda_stream)
        return y, mean, rstd

    def backward(self, x, gamma, beta, mean, rstd, dy, out=None):
        """dict(dx, dgamma, dbeta).  ``out``: the buffers to write; what it
        holds as None is not computed."""
        if not self.training:
            raise ValueError("backward needs training=True")
        self._take_inputs(x, gamma, beta)
        self._take("dy", dy, x.numel(), self.tdtype)
        for what, t in (("mean", mean), ("rstd", rstd)):
            self._take(what, t, self.n * self.groups, torch.float32)
        if out is None:
            out = dict(dx=torch.empty_like(x), dgamma=torch.empty_like(gamma), dbeta=torch.empty_like(beta))
        else:
            for what, like in (("dx", x), ("dgamma", gamma), ("dbeta", beta)):
                if out[what] is not None:
                    self._take(what, out[what], like.numel(), self.tdtype)
        _lib.deft_norm_backward(self.desc, x, gamma, beta, mean, rstd, dy, out["dx"], out["dgamma"], out["dbeta"],
                                self.ws, self.ws_bytes, torch.cuda.current_stream(x.device).cuda_stream)
        return out


_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
