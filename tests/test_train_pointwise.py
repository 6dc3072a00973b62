"""The example's training step: pointwise layers, norm, gradient norm, Muon and AdamW together."""
import importlib.util
import math
import os

import pytest
import torch

from conftest import ROOT
from irregular_gather_cnn_amd import _lib as L
from irregular_gather_cnn_amd.optim import Muon
from irregular_gather_cnn_amd.pointwise import Pointwise8
from oracle import pw8 as O


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_pointwise", os.path.join(ROOT, "examples", "train_pointwise.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["channels_first", "channels_last"])
def test_runs_and_repeats_its_losses(example, layout):
    losses = example.train(steps=6, layout=layout, log=lambda *a: None)
    assert all(math.isfinite(x) for x in losses)
    assert losses == example.train(steps=6, layout=layout, log=lambda *a: None)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["channels_first", "channels_last"])
def test_block_gradients_against_the_formulas(example, layout):
    """The outer layers' gradients, through the whole block, against the formulas in float64 on what the block's
    own calls passed on.  bf16 results: half a step, 2^-8, and the 8-bit sums', 7 * 2^-13 of each group's largest."""
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(5)
    n, c, hidden, s = 2, 72, 200, 150
    block = example.Block(n, c, hidden, s, 8, "gelu", layout, dev)
    params = {k: v.bfloat16() for k, v in block.init(gen).items()}
    grads = {k: torch.zeros_like(v) for k, v in params.items()}
    shape = (n, c, s) if layout == "channels_first" else (n, s, c)
    x, dy = (torch.randn(shape, generator=gen, device=dev).bfloat16() for _ in range(2))
    packed = block.pack(params)
    y, saved = block.forward(x, params, packed)
    block.backward(params, packed, saved, dy, grads)
    saved1, z, mean, rstd, saved2 = saved
    a, _, _ = block.norm.forward(z, params["gamma"], params["beta"])

    def rows(t):
        return (t if layout == "channels_last" else t.transpose(1, 2)).reshape(n * s, -1)

    for what, got, want in (("y", rows(y), O.forward(rows(a), params["w2"], params["b2"])),
                            ("dw2", grads["w2"], O.backward(rows(a), params["w2"], rows(dy))["dw"])):
        exact, mag, group, _ = want
        off, allowed = (got.double() - exact).abs(), 2.0 ** -8 * exact.abs() + 7 * 2.0 ** -13 * group + 2.0 ** -16 * mag
        assert (off <= allowed).all(), what


@pytest.mark.gpu
def test_a_captured_step_of_layer_and_muon():
    """pack, forward, backward, norm and step in one graph, replayed with eager work between."""
    n, c, s, o = 2, 96, 130, 160
    gen = torch.Generator(device="cuda").manual_seed(6)

    def make():
        torch.manual_seed(0)
        master = torch.randn((o, c), generator=torch.Generator(device="cuda").manual_seed(7), device="cuda") * 0.1
        w, g = master.bfloat16(), torch.zeros((o, c), dtype=torch.bfloat16, device="cuda")
        return w, g, Muon([w], [g], masters=[master]), Pointwise8(n, c, s, o, training=True)

    x, dy = (torch.randn(shape, generator=gen, device="cuda").bfloat16() for shape in ((n, c, s), (n, o, s)))

    def step(w, g, opt, layer):
        packed = layer.pack(w)
        y, saved = layer.forward(x, packed)
        out = dict(dx=torch.empty_like(x), dw=g)
        layer.backward(saved, packed, dy, out=out)
        opt.step(control=opt.grad_norm(max_norm=1.0))
        return y, out["dx"]

    captured, eager = make(), make()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            held = step(*captured)
    for k in range(4):
        x.copy_(torch.roll(x, 1, 2))
        dy.mul_(-1.5)
        graph.replay()
        torch.cuda.synchronize()
        want = step(*eager)
        assert all(torch.equal(a, b) for a, b in zip(held, want)), k
        assert torch.equal(captured[0], eager[0]) and torch.equal(captured[2].masters[0], eager[2].masters[0])
        torch.cuda.synchronize()


@pytest.mark.parametrize("current", [0, 1])
def test_new_operators_launch_on_their_tensors_device(current, monkeypatch):
    """Without a GPU: a handle whose tensors are elsewhere makes that device the current one for its calls."""
    import irregular_gather_cnn_amd.optim as optim
    import irregular_gather_cnn_amd.pointwise as pointwise

    entered, now = [], [current]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before = now[0]
            now[0] = self.index
            entered.append(self.index)

        def __exit__(self, *a):
            now[0] = self.before

    for m in (optim, pointwise):
        monkeypatch.setattr(m, "elsewhere", lambda index: now[0] != 0)
        monkeypatch.setattr(m, "current_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    h = Pointwise8(2, 8, 20, 12, layout="channels_last", dtype="f32", training=True, device="cpu")
    w, x, dy = torch.zeros(12, 8), torch.zeros(2, 20, 8), torch.zeros(2, 20, 12)
    opt = Muon([w], [torch.zeros(12, 8)])
    entered.clear()
    called = []

    def fake(*a):
        called.append(now[0])
        return 0

    h._pack = h._forward = h._backward = opt._call = fake
    # on the CPU the index is -1; the fake device 0 stands for it
    h._index = opt.index = opt.grads.index = 0
    monkeypatch.setattr(Pointwise8, "_unfit", lambda self, t, kind: False)
    packed = h.pack(w)
    y, saved = h.forward(x, packed)
    h.backward(saved, packed, dy)
    opt.step()
    assert called == [0] * 4
    assert entered == ([0] * 4 if current else [])


def test_exports_have_their_signatures():
    lib = L.load()
    for name in ("deft_pw8_pack", "deft_pw8_forward", "deft_pw8_backward", "deft_muon_step"):
        assert getattr(lib, name).argtypes and name in L.EXPORTED
