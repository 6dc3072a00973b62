"""The 8-bit pointwise convolution at the ends of its values' range.

Finite values go up to 2^128 - 2^104 and round to codes that stand for 2^128 at most; blocks of tiny values have
the power 2^-127, so their codes' least step is 2^-136.  Products of a factor at one end and one at the other are
ordinary numbers.  Codes and products are exact, so results have the bounds of test_pointwise.py, without what is
allowed there for factors under 2^-126.  fp32: instructions with one of every eight codes in place add the terms one
by one, and each addition may cut 2^-23 of the sum of the magnitudes so far.
"""
import pytest
import torch

from irregular_gather_cnn_amd.pointwise import Pointwise8
from oracle import pw8 as O
from test_pointwise import HALF, LAYOUTS, TYPES, image_of, rows_of

MOST = {"f32": torch.finfo(torch.float32).max, "bf16": torch.finfo(torch.bfloat16).max}


def check(what, got, want, depth, dtype):
    want, mag, group, _ = want
    assert torch.isfinite(want).all() and mag.max() < 2.0 ** 127  # partial sums stay inside fp32
    steps = (depth + min(512, -(-depth // 128)) + 1) * 2.0 ** -23
    allowed = mag * steps + (group * 7 * 2.0 ** -13 if dtype == "bf16" else 0)
    allowed = allowed * (1 + HALF[dtype]) + want.abs() * HALF[dtype] + 2.0 ** -126
    off = (got.double() - want).abs()
    print("  %-3s worst error / bound %.3f" % (what, torch.nan_to_num(off / allowed, 1e9).max().item()), flush=True)
    bad = torch.nonzero(~(off <= allowed))
    assert len(bad) == 0, (what, len(bad), bad[:5].tolist())


def pair(rows, c_in, c_out, dtype, kind, gen):
    """x [rows][c_in] and w [c_out][c_in], normal values but for the blocks (128 channels) of extremes: products
    of all blocks are of like size."""
    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    x, w = rand(rows, c_in), rand(c_out, c_in)
    blocks = [slice(k, k + 128) for k in range(0, c_in, 128)]
    for k, b in enumerate(blocks):
        if kind == "large" and k != 1:
            # up to the type's largest, by signs; some rows only here and there
            x[:, b] = torch.sign(x[:, b]) * (MOST[dtype] * (1 - 0.1 * torch.rand(x[:, b].shape, generator=gen, device="cuda")))
            x[1::3, b] *= (torch.rand(x[1::3, b].shape, generator=gen, device="cuda") < 0.1)
            w[:, b] *= 1e-38
            w[::4, b] = 0
        elif kind == "small" and k != 1:
            x[:, b] *= 1e-39 if k % 2 == 0 else 1e-36
            w[:, b] *= 1e38 if k % 2 == 0 else 1e35
            w[:, b].clamp_(-1.5e38, 1.5e38)
        elif kind == "mixed":
            # per row: a row's blocks have powers of their own, under weights of one size
            size = 10.0 ** (-40 + 60 * torch.rand((rows, 1), generator=gen, device="cuda"))
            x[:, b] *= size
            w[:, b] *= 1e12
    return x.to(TYPES[dtype]), w.to(TYPES[dtype])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["large", "small", "mixed"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,s,c_in,c_out", [(4, 4, 500, 90), (1, 9, 130, 40), (3, 41, 300, 70), (2, 500, 640, 200),
                                            (8, 1100, 200, 1500), (1, 60, 2100, 90), (1, 300, 2100, 90), (1, 50, 140, 33),
                                            (1, 4200, 1000, 4100)])
def test_forward(n, s, c_in, c_out, layout, dtype, kind):
    print("pw8 range", n, s, c_in, c_out, layout, dtype, kind, flush=True)
    x, w = pair(n * s, c_in, c_out, dtype, kind, torch.Generator(device="cuda").manual_seed(1))
    for training in (False, True):
        h = Pointwise8(n, c_in, s, c_out, layout=layout, dtype=dtype, training=training)
        y, _ = h.forward(image_of(x, n, s, layout), h.pack(w))
        check("y", rows_of(y, layout), O.forward(x, w), c_in, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["large", "small", "mixed"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,s,c_in,c_out", [(3, 200, 70, 300), (2, 1030, 40, 30)])
def test_gradients(n, s, c_in, c_out, layout, dtype, kind):
    """dx from extreme dy, dw from extreme dy and x, in blocks of rows."""
    print("pw8 range gradients", layout, dtype, kind, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(2)
    dy, wt = pair(n * s, c_out, c_in, dtype, kind, gen)  # dx sums over c_out
    w = wt.t().contiguous()
    dyt, xt = pair(c_out, n * s, c_in, dtype, kind, gen)  # dw sums over the rows
    h = Pointwise8(n, c_in, s, c_out, layout=layout, dtype=dtype, training=True)
    packed = h.pack(w)
    one = torch.ones((n * s, c_in), dtype=TYPES[dtype], device="cuda")
    _, saved = h.forward(image_of(one, n, s, layout), packed)
    g = h.backward(saved, packed, image_of(dy, n, s, layout), out=dict(dx=torch.empty_like(image_of(one, n, s, layout))))
    check("dx", rows_of(g["dx"], layout), O.backward(one, w, dy)["dx"], c_out, dtype)
    _, saved = h.forward(image_of(xt.t().contiguous(), n, s, layout), packed)
    g = h.backward(saved, packed, image_of(dyt.t().contiguous(), n, s, layout), out=dict(dw=torch.empty_like(w)))
    check("dw", g["dw"], O.backward(xt.t().contiguous(), w, dyt.t().contiguous())["dw"], n * s, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_largest_value_beside_zeros_and_small_weights(dtype, rows):
    """A value that rounds to 2^128: nothing of it reaches outputs whose weight is 0, the others are finite."""
    x = torch.zeros((rows, 256), dtype=TYPES[dtype], device="cuda")
    x[1, 7] = MOST[dtype]
    x[2, 200], x[2, 3] = -MOST[dtype], 1.0
    w = torch.zeros((20, 256), dtype=TYPES[dtype], device="cuda")
    w[0, 7], w[1, 200], w[2, 3] = 1e-10, 2.0 ** -20, 3e-10
    h = Pointwise8(1, 256, rows, 20, layout="channels_last", dtype=dtype)
    y, _ = h.forward(x.view(1, rows, 256), h.pack(w))
    check("y", y.view(rows, 20), O.forward(x, w), 256, dtype)
    assert not y[0, 1, 1:].any() and not y[0, 0].any()
