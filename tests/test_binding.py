"""Arguments of the ctypes binding (irregular_gather_cnn_amd/_lib.py), and the device that calls run on."""
import ctypes
import timeit

import pytest
import torch

from irregular_gather_cnn_amd import _lib as L
from irregular_gather_cnn_amd import _stream
from irregular_gather_cnn_amd.norm import GroupNormAct
from irregular_gather_cnn_amd.optim import AdamW, GradNorm


def test_pointer_arguments():
    t = torch.zeros(3)
    assert L._ptr(t) == t.data_ptr()
    assert L._ptr(None) is None
    assert L._ptr(4096) == 4096
    assert L._ptr(ctypes.c_void_p(64)) == 64
    with pytest.raises(TypeError):
        L._ptr("4096")


def test_plain_addresses_take_no_longer_than_tensors():
    """They did while a tensor was assumed first and the exception caught: 3 times as long; now 0.6."""
    t = torch.zeros(3)

    def best(v):
        return min(timeit.repeat(lambda: L._ptr(v), number=20000, repeat=7))

    assert best(4096) < 1.5 * best(t)
    assert best(None) < 1.5 * best(t)


@pytest.mark.parametrize("current", [0, 1])
def test_operators_launch_on_their_tensors_device(current, monkeypatch):
    """The C functions, replaced here, see the tensors' device (1) as the current one and its stream,
    whatever the program's current device is."""
    now, seen = [current], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *exc):
            now[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(_stream, "_device", lambda: now[0], raising=False)
    monkeypatch.setattr(_stream, "_raw", lambda index: 100 * index)

    def function(*args):
        seen.append((now[0], args[-1]))
        return 0

    there = torch.device("cuda", 1)
    x, c = torch.zeros(2, 8, 4), torch.zeros(8)
    st = torch.zeros(2, 2)
    h = GroupNormAct(2, 8, 4, 2, dtype="f32", training=True, device="cpu")
    h.device, h._index, h._unfit, h._forward, h._backward = there, 1, lambda t, kind: False, function, function
    h.forward(x, c, c)
    h.backward(x, c, c, st, st, x)
    p, g = [torch.zeros(9)], [torch.zeros(9)]
    norm, opt = GradNorm(g), AdamW(p, g)
    for grads in (norm.grads, opt.grads):
        grads.device, grads.index = there, 1
    opt.device = there
    norm._call = opt._call = opt._norm._call = function
    norm()
    opt.grad_norm()
    opt.step()
    assert seen == [(1, 100)] * 5
    assert now[0] == current
    assert opt.steps == 1
