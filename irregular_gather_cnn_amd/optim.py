"""The end of a training step: gradient norm and AdamW over a list of tensors.

PyTorch only supplies device memory and the stream; the arithmetic runs in
libdeft.so (``deft_grad_norm``, ``deft_adamw_step``) through the binding in
``_lib``.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _lib
from ._stream import current_stream, elsewhere

# the fields of a deft_adamw_tensor, packed in a fifth of the time that its ctypes constructor takes
_ITEM = struct.Struct("@7Pqd")
_DTYPES = {torch.float32: _lib.DEFT_F32, torch.bfloat16: _lib.DEFT_BF16}


def _dtype_of(tensors, what):
    kinds = {t.dtype for t in tensors}
    if len(kinds) > 1 or not kinds <= set(_DTYPES):
        raise TypeError("%s must all be float32 or all bfloat16, got %s" % (what, sorted(map(str, kinds))))
    return _DTYPES[kinds.pop()] if kinds else _lib.DEFT_F32


def _dense(t, what, index):
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    if t.get_device() != index:
        raise ValueError("%s is on %s, the first tensor is not" % (what, t.device))


def _hold(tensors):
    """The memory of these tensors, for as long as its addresses are in use, also where a program gives
    a tensor other memory (``t.data = ...``)."""
    return [t.untyped_storage() for t in tensors if t is not None]


class _Gradients:
    """The gradient buffers of a program: their sizes and dtype for good, the
    buffers themselves until :meth:`bind` names others."""

    def __init__(self, grads):
        self.tensors = list(grads)
        if not self.tensors:
            raise ValueError("no gradients")
        self.sizes = [g.numel() for g in self.tensors]
        self.dtype = _dtype_of(self.tensors, "gradients")
        self.device, self.index = self.tensors[0].device, self.tensors[0].get_device()
        self.pointers = (ctypes.c_void_p * len(self.sizes))()
        self.bind(self.tensors)

    def bind(self, grads):
        grads = list(grads)
        if len(grads) != len(self.sizes):
            raise ValueError("%d gradients for %d tensors" % (len(grads), len(self.sizes)))
        for k, (g, n) in enumerate(zip(grads, self.sizes)):
            if g.numel() != n or _DTYPES.get(g.dtype) != self.dtype:
                raise ValueError("gradient %d must have %d elements of the dtype of the first ones" % (k, n))
            _dense(g, "gradient %d" % k, self.index)
        self.tensors, self.held = grads, _hold(grads)
        for k, g in enumerate(grads):
            self.pointers[k] = g.data_ptr()


class GradNorm:
    """Norm of all gradients and the factor that clips them.

    ``grads``: the gradient buffers (device tensors, all float32 or all
    bfloat16), read at every call; :meth:`bind` names others of the same
    sizes.  A call returns the device tensor ``control`` = {norm, factor, 1 if
    all gradients are finite else 0, 0}, valid until the next call; nothing is
    copied to the host."""

    def __init__(self, grads):
        self._setup(_Gradients(grads))

    def _setup(self, grads):
        self.grads = grads
        count = len(grads.sizes)
        self._n = (ctypes.c_int64 * count)(*grads.sizes)
        self.ws_bytes = _lib.deft_grad_norm_workspace_bytes(count)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=grads.device)
        self.control = torch.zeros(4, dtype=torch.float32, device=grads.device)
        # small lists wait for the host: the C function is called without the binding's wrapper
        self._call, self._ws, self._out = _lib.load().deft_grad_norm, self.ws.data_ptr(), self.control.data_ptr()

    def bind(self, grads):
        self.grads.bind(grads)

    def __call__(self, max_norm=float("inf"), inv_scale=1.0):
        g = self.grads
        if elsewhere(g.index):
            with torch.cuda.device(g.index):
                return self(max_norm, inv_scale)
        code = self._call(g.pointers, self._n, len(g.sizes), g.dtype, max_norm, inv_scale, self._out, self._ws,
                          self.ws_bytes, current_stream(g.index))
        if code:
            raise _lib.DeftError(code, "deft_grad_norm")
        return self.control


class AdamW:
    """AdamW with decoupled weight decay over ``params`` (device tensors, all
    float32 or all bfloat16, updated in place) and their gradient buffers
    ``grads`` (likewise; read at every step, :meth:`bind` names others).

    ``bits``: 32 (fp32 states) or 8 (e4m3 codes of m and sqrt(v), one fp32
    scale for each 256 elements).  ``masters``: None, True (fp32 copies of
    bfloat16 params are made and updated, params are their rounded copies) or
    a list of fp32 tensors.  ``weight_decay``: one number or one per tensor.
    ``states``: None (zeros) or a list of (m, v, m_scale, v_scale) per param,
    updated in place (the scales None with 32 bits), as :attr:`states` of an
    earlier run whose :meth:`taken` steps are passed as ``step``.

    The addresses of all tensors are taken here and in :meth:`bind`, and that
    memory is held: a tensor that is given other memory later on (``p.data =
    ...``) needs a new handle, a gradient a new :meth:`bind`."""

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, bits=32,
                 masters=None, states=None, step=0, seed=0):
        self.params = list(params)
        if not self.params:
            raise ValueError("no params")
        if bits not in (8, 32):
            raise ValueError("bits must be 8 or 32, got %r" % (bits,))
        self.device, self.index = self.params[0].device, self.params[0].get_device()
        p_dtype = _dtype_of(self.params, "params")
        for p in self.params:
            _dense(p, "a param", self.index)
        self.sizes = [p.numel() for p in self.params]
        self.grads = _Gradients(grads)
        if self.grads.sizes != self.sizes or self.grads.device != self.device:
            raise ValueError("the gradients' sizes and device must be those of the params")
        if masters is True:
            masters = [p.float() for p in self.params]
        self.masters = list(masters) if masters else None
        if states is None:
            states = [self._zero_state(n, bits) for n in self.sizes]
        self.states = [tuple(s) for s in states]
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * len(self.params)
        for what, got in (("masters", self.masters), ("states", self.states), ("weight decays", decay)):
            if got is not None and len(got) != len(self.params):
                raise ValueError("%d %s for %d params" % (len(got), what, len(self.params)))
        self._check_states(bits)
        self.lr, self.steps, self.seed = lr, int(step), int(seed)
        self._skips = torch.zeros(_lib.DEFT_SKIPS_BYTES // 4, dtype=torch.int32, device=self.device)
        self.skipped = self._skips[:1]
        self._desc = _lib.deft_adamw_desc(p_dtype, self.grads.dtype, bits, 1 if self.masters else 0, 0, lr, betas[0],
                                          betas[1], eps, 0, self._skips.data_ptr())
        packed = []
        for k, p in enumerate(self.params):
            m, v, ms, vs = self.states[k]
            packed.append(_ITEM.pack(p.data_ptr(), self.grads.pointers[k] or 0, m.data_ptr(), v.data_ptr(),
                                     ms.data_ptr() if bits == 8 else 0, vs.data_ptr() if bits == 8 else 0,
                                     self.masters[k].data_ptr() if self.masters else 0, self.sizes[k], decay[k]))
        self._list = (_lib.deft_adamw_tensor * len(packed)).from_buffer_copy(b"".join(packed))
        self._held = _hold(self.params + (self.masters or []) + [t for s in self.states for t in s])
        self._call, self._ref = _lib.load().deft_adamw_step, ctypes.byref(self._desc)
        self._norm = GradNorm.__new__(GradNorm)
        self._norm._setup(self.grads)

    def bind(self, grads):
        """From now on the gradients are read from these tensors."""
        self.grads.bind(grads)
        for item, g in zip(self._list, self.grads.pointers):
            item.g = g

    def _zero_state(self, n, bits):
        if bits == 32:
            return [torch.zeros(n, dtype=torch.float32, device=self.device) for _ in range(2)] + [None, None]
        scales = -(-n // 256)
        return [torch.zeros(n, dtype=torch.uint8, device=self.device).view(torch.float8_e4m3fn) for _ in range(2)] + [
            torch.zeros(scales, dtype=torch.float32, device=self.device) for _ in range(2)]

    def _check_states(self, bits):
        kind = torch.float32 if bits == 32 else torch.float8_e4m3fn
        for k, n in enumerate(self.sizes):
            want = [(t, n, kind, "state %d" % k) for t in self.states[k][:2]]
            if bits == 8:
                want += [(t, -(-n // 256), torch.float32, "scales of state %d" % k) for t in self.states[k][2:]]
            if self.masters:
                want.append((self.masters[k], n, torch.float32, "master %d" % k))
            for t, size, dtype, what in want:
                if t is None or t.numel() != size or t.dtype != dtype:
                    raise ValueError("%s must have %d elements of %s" % (what, size, dtype))
                _dense(t, what, self.index)

    def grad_norm(self, max_norm=float("inf"), inv_scale=1.0):
        """``control`` of the gradients (see :class:`GradNorm`), for :meth:`step`."""
        return self._norm(max_norm, inv_scale)

    def taken(self):
        """How many steps were taken: those counted less those skipped.  Waits for the device."""
        return self.steps - int(self.skipped.item())

    def step_seed(self, step):
        """The seed that rounds the 8-bit states of step number ``step``."""
        return (self.seed + step * 0x9E3779B9) & 0xFFFFFFFF

    def step(self, control=None, lr=None, schedule=None):
        """One step.  ``control``: what :meth:`grad_norm` returned; its factor
        multiplies the gradients and the step writes nothing if they are not
        finite.  :attr:`steps` counts it all the same, as the host does not
        know; the bias corrections of later steps do not (:attr:`skipped`, on
        the device).  ``lr``: from now on.  ``schedule``: 4 device doubles {lr,
        1 - beta1^t, 1 - beta2^t, seed} that the kernels read in place of the
        host's and of that count, for a step captured in a graph."""
        if lr is not None:
            self.lr = lr
        if control is not None or schedule is not None:
            for what, t, kind in (("control", control, torch.float32), ("schedule", schedule, torch.float64)):
                if t is not None and (t.numel() != 4 or t.dtype != kind or t.device != self.device
                                      or not t.is_contiguous()):
                    raise ValueError("%s must be 4 contiguous elements of %s on %s" % (what, kind, self.device))
        if elsewhere(self.grads.index):
            with torch.cuda.device(self.grads.index):
                return self.step(control, lr, schedule)
        d = self._desc
        d.lr, d.step, d.seed = self.lr, self.steps + 1, self.step_seed(self.steps + 1)
        code = self._call(self._ref, self._list, len(self.params), None if control is None else control.data_ptr(),
                          None if schedule is None else schedule.data_ptr(), current_stream(self.grads.index))
        if code:
            raise _lib.DeftError(code, "deft_adamw_step")
        self.steps += 1
