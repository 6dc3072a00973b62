"""Every kernel instance of the group norm against the oracle.

A call's shape, types and activation choose the instance: its form (one
workgroup a group, several that exchange their sums, or read twice), elements
per access, accesses per thread, 1024 threads, and whether the backward keeps
dz.  The shapes below reach every instance that a large sample of shapes does,
which a CPU test holds them to.
"""
import math
import random

import numpy as np
import pytest
import torch

from irregular_gather_cnn_amd import _lib as L
from irregular_gather_cnn_amd.norm import GroupNormAct
from oracle import norm as O
from oracle import norm64 as O64

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ["none", "relu", "silu", "gelu"]
LAYOUTS = ["channels_first", "channels_last"]
FORMS = ["whole", "joint", "twice"]

# (n, c, s, groups), for a device of 256 units
SHAPES = {
    ('channels_first', 'bf16'): [
        (1, 1, 1, 1), (1, 1, 9, 1), (1, 1, 20349, 1), (1, 4, 6413, 1), (1, 18, 517, 1), (1, 18, 1553, 1),
        (1, 77, 261, 1), (1, 1167, 10476, 1), (1, 1770, 5, 1), (2, 1683, 3103, 99), (24, 8400, 17, 8)],
    ('channels_first', 'f32'): [
        (1, 1, 1, 1), (1, 1, 4, 1), (1, 1, 2216354, 1), (1, 3, 2151958, 1), (1, 4, 3188, 1), (1, 11, 1405, 1),
        (1, 34, 466, 1), (1, 555, 4142, 1), (2, 2504, 10, 2), (4, 1248, 1046, 48), (24, 8400, 17, 8)],
    ('channels_last', 'bf16'): [
        (1, 1, 1, 1), (1, 6, 1367, 2), (1, 7, 85995, 7), (1, 8, 1, 8), (1, 9, 1052, 3), (1, 26, 987, 2),
        (1, 77, 261, 1), (1, 113, 1523, 113), (1, 169, 1402, 169), (1, 284, 7385, 71), (2, 4, 262461, 2),
        (3, 26818, 25, 23), (130, 9, 2462, 3), (207, 9, 4395, 3)],
    ('channels_last', 'f32'): [
        (1, 1, 1, 1), (1, 3, 2750, 3), (1, 3, 700874, 3), (1, 4, 1, 1), (1, 5, 1100, 1), (1, 9, 1391, 9),
        (1, 76, 1830, 76), (1, 81, 2438, 81), (1, 284, 7385, 71), (2, 525, 1018, 25), (3, 17115, 41, 15),
        (24, 8400, 17, 8), (87, 5, 4201, 1)],
}


def accesses(cut):
    """Of the kernel, which is built for some numbers."""
    return 16 if cut["vec"] == 1 else next(u for u in (4, 8, 16, 32) if cut["accesses"] <= u)


def instances(layout, dtype, n, c, s, g, act, cus=256):
    d = L.deft_norm_desc(n, c, s, g, L.LAYOUTS[layout], L.ACTIVATIONS[act],
                         L.DEFT_BF16 if dtype == "bf16" else L.DEFT_F32, 1e-5)
    out = set()
    for back in (False, True):
        cut = L.deft_debug_norm_cut(d, back, cus)
        u, form = accesses(cut), FORMS[cut["form"]]
        keep = back and cut["vec"] == 8 and u <= 8 and act in ("silu", "gelu") and form != "twice"
        out.add((back, layout, dtype, cut["vec"], u, form, keep, cut["threads"] == 1024,
                 form == "joint" and bool(cut["direct"])))
    return out


# ------------------------------------------------------------------ CPU

def test_the_shapes_reach_every_instance():
    covered = set()
    for (layout, dtype), shapes in SHAPES.items():
        for shape in shapes:
            for act in ("relu", "gelu"):
                covered |= instances(layout, dtype, *shape, act)
    r = random.Random(5)

    def spread(low, high):
        return max(low, min(high, int(round(math.exp(r.uniform(math.log(low), math.log(high)))))))

    for k in range(40000):
        per, g, n = spread(1, 2048 if k % 4 == 0 else 40), spread(1, 480), spread(1, 600 if k % 3 == 0 else 32)
        s = spread(1, max(1, min(1 << 22, 40_000_000 // (n * per * g))))
        layout, dtype, act = r.choice(LAYOUTS), r.choice(["f32", "bf16"]), r.choice(ACTS)
        assert instances(layout, dtype, n, per * g, s, g, act) <= covered, (layout, dtype, n, per * g, s, g, act)
    # what the cut has by name
    for part in ((True, "channels_last", "f32", 4, 8, "whole", False, True, False),
                 (True, "channels_first", "f32", 4, 8, "whole", False, True, False),
                 (True, "channels_first", "bf16", 8, 8, "whole", False, True, False),
                 (False, "channels_last", "bf16", 8, 32, "whole", False, False, False),
                 (False, "channels_first", "f32", 4, 32, "whole", False, False, False),
                 (True, "channels_last", "bf16", 8, 16, "whole", False, False, False),
                 (True, "channels_last", "bf16", 8, 8, "whole", True, False, False),
                 (True, "channels_first", "bf16", 8, 8, "twice", False, False, False),
                 (False, "channels_first", "f32", 4, 8, "twice", False, False, False),
                 (True, "channels_last", "f32", 1, 16, "twice", False, False, False)):
        assert part in covered, part


@pytest.mark.parametrize("name", ACTS)
def test_the_two_oracles_agree(name):
    r = np.random.default_rng(0)
    n, c, s, g = 2, 12, 37, 3
    x, dy = 2 * r.standard_normal((2, n, c, s))
    gamma, beta = r.standard_normal((2, c))
    t = [torch.from_numpy(v) for v in (x, gamma, beta, dy)]
    f = O.forward(x, gamma, beta, g, 1e-3, name, "f32")
    f64 = O64.forward(t[0], t[1], t[2], g, 1e-3, name, "f32", 4, 4)
    for k in f:
        np.testing.assert_allclose(f64[k][0].numpy(), f[k][0], rtol=1e-13, atol=1e-14)
        assert (f64[k][1].numpy() <= f[k][1]).all()  # of fewer additions
    b = O.backward(x, gamma, beta, f["mean"][0], f["rstd"][0], dy, g, name, "f32")
    b64 = O64.backward(*t[:3], f64["mean"][0], f64["rstd"][0], t[3], g, name, "f32")
    for k in b:
        np.testing.assert_allclose(b64[k][0].numpy(), b[k][0], rtol=1e-12, atol=1e-13)
        np.testing.assert_allclose(b64[k][1].numpy(), b[k][1], rtol=1e-9)


# ------------------------------------------------------------------ GPU

def inputs(layout, dtype, n, c, s, seed=0, offset=0.0):
    """x, gamma, beta, dy on the device, and their values [n][c][s] or [c] in float64."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    x = rand(n, c, s) * (0.5 + rand(c).abs())[:, None] + rand(c)[:, None] + offset
    x, gamma, beta, dy = (v.to(TYPES[dtype]) for v in (x, 1 + 0.3 * rand(c), 0.3 * rand(c), rand(n, c, s)))
    values = [v.double() for v in (x, gamma, beta, dy)]
    if layout == "channels_last":
        x, dy = (v.transpose(1, 2).contiguous() for v in (x, dy))
    return (x, gamma, beta, dy), values


def plain(t, layout):
    return (t.transpose(1, 2) if t.dim() == 3 and layout == "channels_last" else t).double()


def check(got, want, half, what):
    value, bound = want
    bound = bound + half * (value.abs() + bound) + 1e-37
    bad = ~((got - value).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (
        what, bad.sum(), bad.numel(), ((got - value).abs() / bound).max())


def run_both(layout, dtype, n, c, s, g, name, eps=1e-5, seed=0, offset=0.0):
    print("norm", layout, dtype, n, c, s, g, name, flush=True)
    (x, gamma, beta, dy), (xv, gv, bv, dv) = inputs(layout, dtype, n, c, s, seed, offset)
    h = GroupNormAct(n, c, s, g, eps=eps, act=name, layout=layout, dtype=dtype, training=True)
    y, mean, rstd = h.forward(x, gamma, beta)
    cut = L.deft_debug_norm_cut(h.desc, False)
    f = O64.forward(xv, gv, bv, g, eps, name, dtype, accesses(cut), cut["vec"])
    for k, got in (("mean", mean), ("rstd", rstd), ("y", y)):
        check(plain(got, layout), f[k], HALF[dtype if k == "y" else "f32"], k)
    out = h.backward(x, gamma, beta, mean, rstd, dy)
    b = O64.backward(xv, gv, bv, mean.double(), rstd.double(), dv, g, name, dtype)
    for k in ("dx", "dgamma", "dbeta"):
        check(plain(out[k], layout), b[k], HALF[dtype], k)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("layout,dtype,shape", [(*k, v) for k, shapes in SHAPES.items() for v in shapes],
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else v)
def test_instance(layout, dtype, shape, name):
    run_both(layout, dtype, *shape, name)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype,offset", [("f32", 1000.0), ("bf16", 100.0)])
@pytest.mark.parametrize("s", [50, 9001, 90001])
def test_mean_far_from_zero(s, dtype, offset, layout):
    """Groups that one workgroup holds, that several share, and (channels last) that are read twice.  In
    bf16 the bound counts squares about zero: 1e4 of them where a deviation squared is 1."""
    run_both(layout, dtype, 2, 24, s, 3, "silu", seed=5, offset=offset)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("s", [50, 9001, 90001])
def test_sums_of_near_bf16_numbers_are_exact(s, layout):
    """Whole numbers from 192 to 255: a thread's sums of them and of their squares are whole and below
    2^24, so only fp64 and the last roundings touch the statistics."""
    n, c, g = 2, 24, 3
    gen = torch.Generator(device="cuda").manual_seed(6)
    v = (224 + 8 * torch.randn((n, c, s), generator=gen, device="cuda")).round().clamp(192, 255)
    x = (v.transpose(1, 2) if layout == "channels_last" else v).contiguous().bfloat16()
    one = torch.ones(c, dtype=torch.bfloat16, device="cuda")
    _, mean, rstd = GroupNormAct(n, c, s, g, layout=layout).forward(x, one, one)
    xg = v.double().reshape(n, g, -1)
    m = xg.mean(2)
    # each slice's mean is rounded once, and the group's: 2^-24 each
    assert ((mean.double() - m).abs() <= 2.1 * 2.0 ** -24 * m).all()
    r = (xg.var(2, correction=0) + 1e-5).rsqrt()
    # the slices' means are off by 255 * 2^-24 in 8: squared or times the distance of two means, at most
    # 2 * 255 / 8 roundings of the variance, half of them in rstd
    assert ((rstd.double() - r).abs() <= (6 + 255 / 8) * 2.0 ** -24 * r).all()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("s", [60, 30011, 90011])
def test_what_is_not_finite_stays_in_its_group_in_bf16(s, layout, name):
    n, c, g = 2, 24, 3
    (x, gamma, beta, dy), _ = inputs(layout, "bf16", n, c, s, seed=8)
    h = GroupNormAct(n, c, s, g, act=name, layout=layout, training=True)
    y0, mean0, rstd0 = h.forward(x, gamma, beta)
    d0 = h.backward(x, gamma, beta, mean0, rstd0, dy)
    inside = torch.zeros((n, c), dtype=torch.bool, device="cuda")
    inside[1, 8:16] = True  # image 1, group 1
    for bad in (math.nan, math.inf, -math.inf):
        z = x.clone()
        (z[1, :, 9] if layout == "channels_last" else z[1, 9])[s // 2] = bad
        y, mean, rstd = h.forward(z, gamma, beta)
        d = h.backward(z, gamma, beta, mean, rstd, dy)
        for got, ref in ((y, y0), (d["dx"], d0["dx"])):
            got, ref = plain(got, layout), plain(ref, layout)
            assert torch.equal(got[~inside], ref[~inside])
            assert got[inside].isnan().all()
        assert torch.equal(d["dgamma"].isnan(), inside[1])
