"""Group norm at the ends of its range: rows of 2^31 - 1 positions, whose index
arithmetic passes 32 bits, launches near 2^32 threads, and workspaces that were not zeroed.
"""
import ctypes
import time

import numpy as np
import pytest
import torch

from irregular_gather_cnn_amd import _lib as L
from irregular_gather_cnn_amd.norm import GroupNormAct

H = 2.0 ** -24


@pytest.mark.parametrize("n,c,s,groups,layout,code", [
    # a workgroup of 64 threads for each group, or each band of 16: 2^32 threads are too many
    (2 ** 26 - 1, 1, 1, 1, 0, 0), (2 ** 26, 1, 1, 1, 0, -10), (1, 2 ** 26 - 1, 1, 2 ** 26 - 1, 0, 0),
    (1, 2 ** 26, 1, 2 ** 26, 0, -10), (2 ** 26 - 1, 1, 1, 1, 1, 0), (2 ** 26, 1, 1, 1, 1, -10),
    # 31 groups in a band: numbers of groups past 31 bits
    (2 ** 26 - 1, 31, 1, 31, 1, 0), (2 ** 26 - 1, 62, 1, 62, 1, -10),
    (2 ** 31 - 1, 1, 1, 1, 0, -10), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 0, -10),
    # many channels take no more threads than their groups
    (1, 2 ** 27, 1, 2 ** 16, 0, 0), (1, 2 ** 27, 1, 2 ** 16, 1, 0)])
def test_launches_stay_below_2_32_threads(n, c, s, groups, layout, code):
    d = L.deft_norm_desc(n, c, s, groups, layout, 0, L.DEFT_BF16, 1e-5)
    assert L.load().deft_norm_desc_validate(ctypes.byref(d)) == code


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["channels_last", "channels_first"])
def test_more_channels_than_one_launch_sums(layout):
    """2^27 channels in groups of 2048, one position: dbeta = dy and dgamma = dy h, each rounded once."""
    c, per = 2 ** 27, 2048
    print("norm", layout, c, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, dy = (torch.randn((1, c), generator=gen, device="cuda").bfloat16() for _ in range(2))
    gamma, beta = torch.ones(c, dtype=torch.bfloat16, device="cuda"), torch.zeros(c, dtype=torch.bfloat16, device="cuda")
    h = GroupNormAct(1, c, 1, c // per, layout=layout, training=True)
    _, mean, rstd = h.forward(x, gamma, beta)
    fill = torch.full_like(gamma, 7)
    out = h.backward(x, gamma, beta, mean, rstd, dy, out=dict(dx=None, dgamma=fill, dbeta=fill.clone()))
    assert torch.equal(out["dbeta"], dy.view(-1))
    want = dy.view(-1, per).double() * ((x.view(-1, per).double() - mean.view(-1, 1)) * rstd.view(-1, 1).double())
    assert ((out["dgamma"].view(-1, per).double() - want).abs() <= want.abs() * (2.0 ** -8 + 8 * H)).all()
    # no positions: zeros
    h = GroupNormAct(1, c, 0, c // per, layout=layout, training=True)
    none = torch.empty((1, c, 0), dtype=torch.bfloat16, device="cuda")
    out = h.backward(none, gamma, beta, mean, rstd, none, out=dict(dx=None, dgamma=fill, dbeta=fill.clone()))
    assert not out["dgamma"].any() and not out["dbeta"].any()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["channels_last", "channels_first"])
@pytest.mark.parametrize("s", [2 ** 31 - 1, 2 ** 31 - 9000])
def test_rows_of_the_greatest_length(layout, s):
    """One channel of s positions, summed in float64.  x and dy differ from zero only in the first and last `w` positions,
    so few values are summed, and every output elsewhere is one known number."""
    print("norm", layout, s, flush=True)
    w, guard = 40000, 64
    assert s > 4 * w
    gen = torch.Generator(device="cuda").manual_seed(1)

    def row(fill):
        # 64 elements before and after, so that an access outside the row is seen and stays in memory
        buf = torch.full((s + 2 * guard,), fill, dtype=torch.bfloat16, device="cuda")
        return buf, buf[guard:guard + s]

    xb, x = row(0.0)
    db, dy = row(0.0)
    for t in (x, dy):
        t[:w].normal_(generator=gen)
        t[s - w:].normal_(generator=gen)
    yb, y = row(7.0)
    gb, dx = row(7.0)
    gamma = torch.full((1,), 1.25, dtype=torch.bfloat16, device="cuda")
    beta = torch.full((1,), 0.25, dtype=torch.bfloat16, device="cuda")
    shape = (1, s, 1) if layout == "channels_last" else (1, 1, s)
    h = GroupNormAct(1, 1, s, 1, eps=1e-5, layout=layout, training=True)
    _, mean, rstd = h.forward(x.view(shape), gamma, beta, y=y.view(shape))
    out = h.backward(x.view(shape), gamma, beta, mean, rstd, dy.view(shape),
                     out=dict(dx=dx.view(shape), dgamma=torch.empty_like(gamma), dbeta=torch.empty_like(beta)))

    def ends(t):
        return torch.cat([t[:w], t[s - w:]]).double().cpu().numpy()

    xe, de = ends(x), ends(dy)
    m, r = mean.item(), rstd.item()
    # statistics: fp32 chains of at most 256 in a thread, fp64 beyond
    want = xe.sum() / s
    e_mean = 256 * H * np.abs(xe).sum() / s + H * abs(want)
    assert abs(m - want) <= e_mean
    var = (xe * xe).sum() / s - want * want
    assert abs(r - (var + 1e-5) ** -0.5) <= r * (0.5 * 264 * H * var / (var + 1e-5) + 4 * H)
    # y = 1.25 (x - mean) rstd + 0.25; bf16's rounding, and a few of fp32 before it
    z = 1.25 * (xe - m) * r + 0.25
    ez = 8 * H * (1.25 * (np.abs(xe) + abs(m)) * r + 0.25)
    assert (np.abs(ends(y) - z) <= ez + 2.0 ** -8 * (np.abs(z) + ez)).all()
    # gradients
    hh = (xe - m) * r
    a, b = de.sum(), (de * hh).sum()
    ea, eb = 256 * H * np.abs(de).sum(), 264 * H * np.abs(de * hh).sum()
    for got, value, e in ((out["dbeta"], a, ea), (out["dgamma"], b, eb)):
        assert abs(got.item() - value) <= e + 2.0 ** -8 * (abs(value) + e)
    d = r * (1.25 * de - 1.25 * a / s - hh * 1.25 * b / s)
    ed = 16 * H * r * (1.25 * np.abs(de) + 1.25 * abs(a) / s + np.abs(hh) * 1.25 * abs(b) / s) \
        + r * 1.25 / s * (ea + np.abs(hh) * eb)
    assert (np.abs(ends(dx) - d) <= ed + 2.0 ** -8 * (np.abs(d) + ed)).all()
    # between the ends x and dy are zero: one value each, and every position was written
    for t, value in ((y, 1.25 * (0 - m) * r + 0.25), (dx, r * 1.25 / s * (-a + m * r * b))):
        mid = t[w:s - w]
        assert mid.min() == mid.max()
        if t is dx:
            e = r * 1.25 / s * (ea + abs(m) * r * eb + 16 * H * (abs(a) + abs(m * r * b)))
        else:
            e = 8 * H * (abs(value) + 0.5)
        assert abs(mid[0].item() - value) <= e + 2.0 ** -8 * (abs(value) + e) + 1e-37
    for buf, fill in ((yb, 7.0), (gb, 7.0)):
        assert (buf[:guard] == fill).all() and (buf[guard + s:] == fill).all()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["channels_last", "channels_first"])
@pytest.mark.parametrize("n,c,s,g", [(1, 64, 20001, 1), (2, 40, 9001, 20), (1, 1920, 700, 480)])
def test_a_workspace_that_was_not_zeroed_ends_every_wait(n, c, s, g, layout):
    """The counters of calls begin between two calls, so the workgroups of one call carry two numbers and
    look for words that others replace.  Each element is right or NaN, and the calls end: 24 of them, each
    with two waits of 2 ms and a last one of 10 ms a workgroup at most, a few workgroups after the other."""
    print("norm", n, c, s, g, layout, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(2)
    shape = (n, s, c) if layout == "channels_last" else (n, c, s)
    x, dy = (torch.randn(shape, generator=gen, device="cuda").bfloat16() for _ in range(2))
    gamma, beta = (torch.randn((c,), generator=gen, device="cuda").bfloat16() for _ in range(2))
    good = GroupNormAct(n, c, s, g, act="silu", layout=layout, training=True)
    want = good.forward(x, gamma, beta)
    back = good.backward(x, gamma, beta, want[1], want[2], dy)
    h = GroupNormAct(n, c, s, g, act="silu", layout=layout, training=True)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for fill in (1, 2, 3, 7):
        for _ in range(3):
            h.ws.view(torch.int64).fill_(fill)
            got = h.forward(x, gamma, beta)
            for a, b in zip(got, want):
                assert ((a == b) | a.isnan()).all()
            out = h.backward(x, gamma, beta, want[1], want[2], dy)
            assert ((out["dx"] == back["dx"]) | out["dx"].isnan()).all()
    assert time.perf_counter() - start < 20


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
def test_no_positions_have_no_statistics(given):
    x, c = torch.empty(3, 8, 0, device="cuda"), torch.ones(8, device="cuda")
    h = GroupNormAct(3, 8, 0, 2, dtype="f32")
    torch.full((3, 2), 5.0, device="cuda")  # what memory that is not written is likely to hold
    out = dict(mean=torch.ones(3, 2, device="cuda"), rstd=torch.ones(3, 2, device="cuda")) if given else {}
    y, mean, rstd = h.forward(x, c, c, **out)
    assert y.shape == x.shape and mean.shape == rstd.shape == (3, 2)
    assert mean.isnan().all() and rstd.isnan().all()


def test_backward_refuses_unknown_buffers_before_any_launch():
    x, c, st = torch.zeros(2, 8, 4), torch.ones(8), torch.zeros(2, 2)
    h = GroupNormAct(2, 8, 4, 2, dtype="f32", training=True, device="cpu")
    with pytest.raises(ValueError, match="dw"):
        h.backward(x, c, c, st, st, x, out=dict(dx=x.clone(), dw=c))
    with pytest.raises(ValueError, match="dgamma"):
        h.backward(x, c, c, st, st, x, out=dict(dgamma=x))


@pytest.mark.gpu
def test_backward_writes_the_buffers_it_is_given():
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, dy = (torch.randn((2, 8, 40), generator=gen, device="cuda") for _ in range(2))
    c = torch.randn((8,), generator=gen, device="cuda")
    h = GroupNormAct(2, 8, 40, 2, act="silu", dtype="f32", training=True)
    _, mean, rstd = h.forward(x, c, c)
    want = h.backward(x, c, c, mean, rstd, dy)
    for keep in (("dx",), ("dgamma", "dbeta"), ("dbeta",), ()):
        out = h.backward(x, c, c, mean, rstd, dy, out={k: torch.zeros_like(want[k]) for k in keep})
        assert sorted(out) == sorted(keep)
        for k in keep:
            assert torch.equal(out[k], want[k])
