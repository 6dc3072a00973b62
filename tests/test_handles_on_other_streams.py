"""Handles that go out of use while their calls are still under way on another stream than the one they were made on:
their workspaces stay theirs until the calls have ended."""
import pytest
import torch

from irregular_gather_cnn_amd.optim import Muon
from irregular_gather_cnn_amd.pointwise import Pointwise8


def rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def take(size):
    """What the current stream's next allocations of that size hold: all of them are overwritten."""
    return [torch.full((size,), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(4)]


@pytest.mark.gpu
def test_pointwise():
    x, w, b, dy = rand(2, 256, 500).bfloat16(), rand(300, 256, seed=1).bfloat16(), rand(300, seed=2).bfloat16(), rand(2, 300, 500, seed=3).bfloat16()

    def made():
        return Pointwise8(2, 256, 500, 300, training=True)

    def run(h):
        packed = h.pack(w)
        y, saved = h.forward(x, packed, b)
        return [y] + list(h.backward(saved, packed, dy).values())

    want = run(made())
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    h = made()
    size, at = h.ws.numel(), h.ws.data_ptr()
    with torch.cuda.stream(other):
        torch.cuda._sleep(200_000_000)
        got = run(h)
    del h
    taken = take(size)
    assert at not in [t.data_ptr() for t in taken]
    other.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    assert all((t == 0x7f).all() for t in taken)


@pytest.mark.gpu
def test_muon():
    shapes = [(300, 200), (90, 400)]
    grads = [rand(*s, seed=4 + k) for k, s in enumerate(shapes)]

    def made():
        return Muon([torch.zeros(s, device="cuda") for s in shapes], grads)

    def step(opt):
        opt.step(control=opt.grad_norm(max_norm=0.5))
        return [p for p in opt.params]

    want = step(made())
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    opt = made()
    owned = [opt.ws, opt._norm.ws, opt._norm.control] + opt.states
    sizes, at = [t.numel() * t.element_size() for t in owned], {t.data_ptr() for t in owned}
    del owned
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(200_000_000)
        got = step(opt)
    del opt
    taken = [t for size in sizes for t in take(size)]
    assert not at & {t.data_ptr() for t in taken}
    other.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    assert all((t == 0x7f).all() for t in taken)
