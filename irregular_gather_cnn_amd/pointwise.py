"""Pointwise (1x1) convolution in 8 bits, with its gradients.

PyTorch only supplies device memory and the stream; the arithmetic runs in
libdeft.so (``deft_pw8_pack``, ``deft_pw8_forward``, ``deft_pw8_backward``)
through the binding in ``_lib``.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib
from ._stream import Lent, current_stream, elsewhere


class Pointwise8:
    """y[r][o] = sum_k x[r][k] w[o][k] + b[o] over the n * s positions r, the
    factors rounded to e4m3 with a power of two for each block of 128 values
    (of a row's channels, or of 128 x 128 weights; include/deft.h has the
    formulas).  Sums are fp32.

    ``layout``: "channels_first" (x is [n][c_in][s], such as the
    [n][c][h][w] that :class:`layer.DeformConv` writes, s = h * w, and y is
    [n][c_out][s]) or "channels_last" ([n][s][c_in], [n][s][c_out]).
    ``dtype``: "bf16" or "f32", of all tensors.  ``training``: pack the
    weights, and save what the forward read, for :meth:`backward` too.  Without
    it, calls of at most 16 positions take one launch.

    Calls run on the current stream of their device, whichever device is the
    current one; calls of one handle on several streams must be ordered by the
    caller, as they share the workspace."""

    def __init__(self, n, c_in, s, c_out, layout="channels_first", dtype="bf16", training=False, device="cuda"):
        for what, value, known in (("layout", layout, _lib.LAYOUTS), ("dtype", dtype, _DTYPES)):
            if value not in known:
                raise ValueError("%s must be one of %s, got %r" % (what, sorted(known), value))
        self.desc = _lib.deft_pw8_desc(n, s, c_in, c_out, _lib.LAYOUTS[layout],
                                       _lib.DEFT_BF16 if dtype == "bf16" else _lib.DEFT_F32, 1 if training else 0)
        self._index = torch.empty(0, device=device).get_device()
        with torch.cuda.device(self._index) if elsewhere(self._index) else contextlib.nullcontext():
            _lib.deft_pw8_desc_validate(self.desc)
            self.ws_bytes = _lib.deft_pw8_workspace_bytes(self.desc)
        self.packed_bytes = _lib.deft_pw8_packed_bytes(self.desc)
        self.saved_bytes = _lib.deft_pw8_saved_bytes(self.desc)
        self.n, self.c_in, self.s, self.c_out, self.layout = n, c_in, s, c_out, layout
        self.tdtype, self.training = _DTYPES[dtype], bool(training)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=device)
        self.device, self._lent = self.ws.device, Lent(self._index, [self.ws])
        # what each argument must be: elements and dtype
        x, y, t = n * s * c_in, n * s * c_out, self.tdtype
        self._kinds = dict(x=(x, t), dx=(x, t), y=(y, t), dy=(y, t), w=(c_in * c_out, t), dw=(c_in * c_out, t),
                           b=(c_out, t), db=(c_out, t), weights=(self.packed_bytes, torch.uint8),
                           saved=(self.saved_bytes, torch.uint8))
        self._y_shape = (n, c_out, s) if layout == "channels_first" else (n, s, c_out)
        self._x_shape = (n, c_in, s) if layout == "channels_first" else (n, s, c_in)
        # small calls wait for the host: the C functions are called without the binding's wrappers
        lib, self._ref, self._ws = _lib.load(), ctypes.byref(self.desc), self.ws.data_ptr()
        self._pack, self._forward, self._backward = lib.deft_pw8_pack, lib.deft_pw8_forward, lib.deft_pw8_backward

    def _unfit(self, t, kind):
        return (t.numel() != kind[0] or t.dtype is not kind[1] or t.get_device() != self._index
                or not t.is_contiguous())

    def _refuse(self, **tensors):
        for what, t in tensors.items():
            if t is not None and self._unfit(t, self._kinds[what]):
                raise ValueError("%s must be %d contiguous elements of %s on %s" % (
                    (what,) + self._kinds[what] + (self.device,)))

    def _empty(self, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def pack(self, w, out=None):
        """The codes of w, [c_out][c_in] in any shape of as many elements, as :meth:`forward` and
        :meth:`backward` take them until w changes.  They serve every handle of these channels and this
        ``training``."""
        self._refuse(w=w, weights=out)
        if out is None:
            out = self._empty(self.packed_bytes, torch.uint8)
        if elsewhere(self._index):
            with torch.cuda.device(self._index):
                return self.pack(w, out)
        code = self._pack(self._ref, w.data_ptr(), out.data_ptr(), current_stream(self._index))
        if code:
            raise _lib.DeftError(code, "deft_pw8_pack")
        return out

    def forward(self, x, weights, b=None, y=None, saved=None):
        """(y, saved); ``saved`` is what :meth:`backward` needs of x, None without ``training``."""
        unfit, kinds = self._unfit, self._kinds
        if unfit(x, kinds["x"]) or unfit(weights, kinds["weights"]) or b is not None and unfit(b, kinds["b"]):
            self._refuse(x=x, weights=weights, b=b)
        if y is not None or saved is not None:
            if not self.training and saved is not None:
                raise ValueError("saved needs training=True")
            self._refuse(y=y, saved=saved)
        if y is None:
            y = self._empty(self._y_shape, self.tdtype)
        if self.training and saved is None:
            saved = self._empty(self.saved_bytes, torch.uint8)
        if elsewhere(self._index):
            with torch.cuda.device(self._index):
                return self.forward(x, weights, b, y, saved)
        code = self._forward(self._ref, x.data_ptr(), weights.data_ptr(), None if b is None else b.data_ptr(),
                             y.data_ptr(), None if saved is None else saved.data_ptr(), self._ws, self.ws_bytes,
                             self._lent.to(current_stream(self._index)))
        if code:
            raise _lib.DeftError(code, "deft_pw8_forward")
        return y, saved

    def backward(self, saved, weights, dy, out=None):
        """dict(dx, dw, db) at dy, with what :meth:`forward` saved and the weights that it used.  ``out``: the
        buffers to write; what it leaves out or holds as None is not computed."""
        if not self.training:
            raise ValueError("backward needs training=True")
        self._refuse(saved=saved, weights=weights, dy=dy)
        if out is None:
            out = dict(dx=self._empty(self._x_shape, self.tdtype), dw=self._empty((self.c_out, self.c_in), self.tdtype),
                       db=self._empty(self.c_out, self.tdtype))
        elif not out.keys() <= _GRADIENTS:
            raise ValueError("out may hold %s, got %s" % (sorted(_GRADIENTS), sorted(out)))
        else:
            self._refuse(**out)
        dx, dw, db = out.get("dx"), out.get("dw"), out.get("db")
        if elsewhere(self._index):
            with torch.cuda.device(self._index):
                return self.backward(saved, weights, dy, out)
        code = self._backward(self._ref, saved.data_ptr(), weights.data_ptr(), dy.data_ptr(),
                              None if dx is None else dx.data_ptr(), None if dw is None else dw.data_ptr(),
                              None if db is None else db.data_ptr(), self._ws, self.ws_bytes,
                              self._lent.to(current_stream(self._index)))
        if code:
            raise _lib.DeftError(code, "deft_pw8_backward")
        return out


_GRADIENTS = {"dx", "dw", "db"}
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
