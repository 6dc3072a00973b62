"""Muon's products by tiles of 128 and 256: pairs of fp16 as near as steps in fp32, bf16 weights bit for bit.

Pairs hold 22 bits where fp32 holds 24, so directions may be 4 times as far from the 64-bit ones as those of steps
in fp32 torch are, and 2^-22 of their size for the first rounding.  That bound is under what one lost part leaves:
the CPU tests plant such losses in an emulation of the steps.  (32 * 2^-22 of the sizes that
test_muon.py's bound adds up over the steps lets a lost part pass at these shapes.)

The lists: which tiles they take on 256 compute units, for Gram products (split over n, or not), squares and
products with X.
"""
import math

import pytest
import torch

from irregular_gather_cnn_amd.optim import Muon
from oracle import muon as O
from test_muon import direction, rand

LISTS = {
    "128, 64, 128": [(1024, 1100), (600, 2300), (1500, 700)],
    "256, 128, 256": [(1100, 4003), (4003, 1100), (1213, 5000)],
    "256, 128, 128": [(2100, 2049)],
    "128, 64, 256": [(300, 5000)] * 5 + [(5001, 300)] * 4,
    "256 not split, 128, 256": [(6000, 6100)],
}


def steps_in_fp32(u, steps=5, part=lambda t, where: t):
    """X after single steps in fp32; part rounds what goes into the products."""
    x = u / torch.linalg.vector_norm(u.double()).float()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t().contiguous()
    for k in range(steps):
        h = part(x, "gram")
        g = h @ h.t()
        h = part(g, "square")
        q = O.B * g + O.C * (h @ h)
        q.diagonal().add_(O.A)
        x = part(q, "left") @ part(x, "right")
    return x.t() if tall else x


def bound(u, want):
    plain = float((steps_in_fp32(u).double() - want).norm())
    return plain, 4 * plain + 2.0 ** -22 * float(want.norm())


def matrix(shape, kind, seed):
    """Normal values, or few strong directions in noise, as gradients have."""
    m, n = shape
    if kind == "normal":
        return rand(shape, seed)
    k = max(1, min(m, n) // 8)
    return rand((m, k), seed) @ rand((k, n), seed + 1000) / math.sqrt(k) + 0.05 * rand(shape, seed + 2000)


# ------------------------------------------------------------------ CPU: the bound notices what it is for

def pairs(t, high, low=True):
    """t times a power of two as one fp16, or as the sum of two."""
    scale = 2.0 ** (14 - math.ceil(math.log2(max(1.0, float(t.abs().max())))))
    v = t * scale
    hi = v.half().float()
    return (hi + (v - hi).half().float() if low else hi) / scale


@pytest.mark.parametrize("shape", [(64, 300), (300, 1000), (500, 400), (600, 2300)])
@pytest.mark.parametrize("kind", ["normal", "strong"])
def test_the_bound_lets_pairs_pass_and_single_parts_not(shape, kind):
    gen = torch.Generator().manual_seed(3)
    m, n = shape
    u = torch.randn(shape, generator=gen)
    if kind == "strong":
        k = min(shape) // 8
        u = torch.randn((m, k), generator=gen) @ torch.randn((k, n), generator=gen) / math.sqrt(k) + 0.05 * u
    want, _ = O.orthogonal(u, 5)
    plain, allowed = bound(u, want)

    def off(part):
        return float((steps_in_fp32(u, part=part).double() - want).norm())

    assert off(lambda t, where: pairs(t, True)) <= allowed
    for lost in (("gram",), ("square",), ("left",), ("right",)):
        assert off(lambda t, where: pairs(t, True, where not in lost)) > allowed, lost


# ------------------------------------------------------------------ GPU

@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["normal", "strong"])
@pytest.mark.parametrize("tiles", LISTS)
def test_directions_are_as_near_as_steps_in_fp32(tiles, kind):
    us = [matrix(s, kind, 10 * k + 1) for k, s in enumerate(LISTS[tiles])]
    print("muon tiles", tiles, kind, flush=True)
    for u, x in zip(us, direction(us)):
        want, _ = O.orthogonal(u, 5)
        plain, allowed = bound(u, want)
        off = float((x.double() - want).norm())
        print("  %s off %.2e, steps in fp32 %.2e, allowed %.2e" % (tuple(u.shape), off, plain, allowed), flush=True)
        assert off <= allowed
        del want
    torch.cuda.empty_cache()


def guarded(t, dtype):
    """A copy of t with 64 elements behind it, and the whole."""
    whole = torch.full((t.numel() + 64,), 7.0, dtype=dtype, device="cuda")
    whole[:t.numel()] = t.flatten()
    return whole[:t.numel()].view(t.shape), whole


@pytest.mark.gpu
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("p_type,g_type,master", [("bf16", "bf16", True), ("bf16", "bf16", False), ("bf16", "f32", True),
                                                  ("f32", "bf16", False)])
@pytest.mark.parametrize("tiles", ["128, 64, 128", "256, 128, 256", "256, 128, 128", "128, 64, 256"])
def test_weights_and_momentum_bit_for_bit(tiles, p_type, g_type, master, nesterov):
    """A step from zero fp32 weights gives the direction, whose bits do not depend on the weights: they are compared
    with the formula on it.  A step that control skips comes before."""
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    shapes = LISTS[tiles]
    print("muon tiles", tiles, p_type, g_type, master, nesterov, flush=True)
    full = [rand(s, 300 + k, 0.05) for k, s in enumerate(shapes)]
    p = [guarded(t, types[p_type]) for t in full]
    masters = [guarded(t, torch.float32) for t in full] if master else None
    g = [matrix(s, "strong", 20 * k + 7).mul_(1e-3).to(types[g_type]) for k, s in enumerate(shapes)]
    m = [guarded(rand(s, 400 + k, 1e-3), torch.float32) for k, s in enumerate(shapes)]
    decay = [0.1 * k for k in range(len(shapes))]
    hyper = dict(momentum=0.9, nesterov=nesterov)
    opt = Muon([t for t, _ in p], g, lr=0.03, weight_decay=decay, masters=[t for t, _ in masters] if master else None,
               states=[t for t, _ in m], adjust="rms", **hyper)
    before = [[t.clone() for t, _ in part] for part in (p, m, masters or [])]

    value = g[-1][3, 3].item()
    g[-1][3, 3] = math.inf
    opt.step(control=opt.grad_norm(max_norm=0.5))
    for part, kept in zip((p, m, masters or []), before):
        assert all(torch.equal(t, k) for (t, _), k in zip(part, kept))
    g[-1][3, 3] = value

    zero = [torch.zeros(s, device="cuda") for s in shapes]
    probe = Muon(zero, g, lr=1.0, weight_decay=0.0, states=[t.clone() for t in before[1]], adjust="none", **hyper)
    control = opt.grad_norm(max_norm=0.5)
    opt.step(control=control)
    probe.step(control=control)
    for k, (rows, cols) in enumerate(shapes):
        mom, u = O.momentum(before[1][k], g[k], 0.9, nesterov, control[1])
        assert torch.equal(m[k][0], mom) and torch.equal(probe.states[k], mom)
        x, _ = O.orthogonal(u, 5)
        assert float((-zero[k].double() - x).norm()) <= bound(u, x)[1]
        want = O.update(before[2][k] if master else before[0][k], -zero[k], 0.03, decay[k], 0.2 * math.sqrt(max(rows, cols)))
        if master:
            assert torch.equal(masters[k][0], want)
        assert torch.equal(p[k][0], want.to(types[p_type]))
    for _, whole in p + m + (masters or []):
        assert (whole[-64:] == 7).all()
    torch.cuda.empty_cache()
