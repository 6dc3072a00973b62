"""The 8-bit pointwise convolution (deft_pw8_*).

CPU: the oracle, and every refusal of the C ABI and of the Python class.  GPU:
against the oracle in float64.

Bounds.  Codes are exact, and so are products of two coded values.  fp32
results: a product's sum takes four instructions of 16 terms for each 64, each
of which may round a sum of the magnitudes so far by 2^-23 (half a step would
be 2^-24), and one addition for each split of its depth: (depth / 16 + splits +
1) 2^-23 of the sum of magnitudes, the 1 for the bias.  There are at most 512
splits, and never more than the depth's blocks of 128.

bf16 results: 8-bit instructions cut 7 terms of each 8 off 13 bits below the
largest one's leading bit.  So a group of 8 is off by at most 7 * 2^-13 of its
largest magnitude, and these errors have no sign in common, so that a result's
are spread as sqrt(7 / 3) 2^-13 of the root of the sum of the largest squares at
most, over many results: both are checked.  With a single large term in each
group the first is reached.

The result is rounded once: half a step of its type.  db sums 128 rows in fp32
in chains of at most 16, then in fp64: 16 * 2^-24 of the magnitudes, and the
rounding of the sum to fp32 and to its type.  Everything below 2^-126 may be
lost on the way, from factors too: 2^-120 is added for it.  Where the sum of
magnitudes passes 2^127, a partial sum in fp32 may pass its range, 2^128, and
every value may come of it: a sum of terms of both signs is infinite, then NaN.
"""
import ctypes

import numpy as np
import pytest
import torch

from irregular_gather_cnn_amd import _lib as L
from irregular_gather_cnn_amd.pointwise import Pointwise8
from oracle import optim as O8
from oracle import pw8 as O

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LAYOUTS = ["channels_first", "channels_last"]


# ------------------------------------------------------------------ CPU: oracle

def test_nearest_is_e4m3():
    r = np.random.default_rng(0)
    t = np.concatenate([r.uniform(-448, 448, 20000), r.standard_normal(20000) * 0.01, O8.e4m3_values(),
                        (O8.e4m3_values()[1:] + O8.e4m3_values()[:-1]) / 2])
    want = O8.decode(O8.encode_nearest(t))
    np.testing.assert_array_equal(O.nearest(torch.from_numpy(t)).numpy(), want)
    f = torch.from_numpy(t).float()
    assert torch.equal(O.nearest(f.double()).float(), f.to(torch.float8_e4m3fn).float())


def test_powers():
    most = torch.tensor([448.0, 448.0 * (1 + 2.0 ** -23), 1.0, 0.0, 1.75, 1.7500001, 2.0 ** -140, 3.4e38, 449.0],
                        dtype=torch.float64)
    e = O.powers(most)
    assert e.tolist() == [0, 1, -8, -127, -8, -7, -127, 120, 1]


def test_a_blocks_values_share_a_power():
    t = torch.zeros((2, 260), dtype=torch.float64)
    t[0, 0], t[0, 127], t[0, 128], t[1, 259] = 448, 2.0 ** -9, 2.0 ** -9 * 1.5, 1000
    t[0, 129] = 2.0 ** -10 * 0.99
    c = O.coded(t)
    assert c[0, 0] == 448 and c[0, 127] == 2.0 ** -9 and c[0, 128] == t[0, 128] and c[1, 259] == 1024
    tile = O.coded(t, 128, 128)
    assert tile[0, 128] == t[0, 128] and tile[0, 127] == 2.0 ** -9


def test_oracle_product_and_gradients_are_linear_maps_of_coded_values():
    """Values that are codes already: the formulas are the plain convolution's and torch's gradients."""
    r = np.random.default_rng(1)

    def codes(*shape):
        # e4m3 values of at most 240, with 256 in each block of 128, so that every scale is 1
        v = O8.decode(r.integers(0, 0x78, shape).astype(np.uint8)) * r.choice([-1.0, 1.0], shape)
        return torch.from_numpy(v)

    x, w, dy = codes(256, 128), codes(128, 128), codes(256, 128)
    for t in (x, w, dy):
        t[::128, :] = 256.0
        t[:, ::128] = 256.0
    b = torch.linspace(-1, 1, 128, dtype=torch.float64)
    xt, wt, bt = (t.clone().requires_grad_() for t in (x, w, b))
    y = torch.nn.functional.linear(xt, wt, bt)
    y.backward(dy)
    assert torch.equal(O.forward(x, w, b)[0], y.detach())
    g = O.backward(x, w, dy)
    assert torch.equal(g["dx"][0], xt.grad) and torch.equal(g["dw"][0], wt.grad) and torch.equal(g["db"][0], bt.grad)


def test_oracle_keeps_what_is_not_finite_apart():
    x = torch.ones((3, 200), dtype=torch.float64)
    w = torch.ones((130, 200), dtype=torch.float64)
    x[1, 5], w[129, 7] = float("inf"), float("nan")
    y = O.forward(x, w)[0]
    bad = torch.isnan(y)
    assert bad[1].all() and bad[:, 129].all() and bad.sum() == 130 + 3 - 1


# ------------------------------------------------------------------ CPU: refusals

FAKE = 0x10000


def desc(n=2, s=100, c_in=32, c_out=48, layout=1, dtype=1, training=1):
    return L.deft_pw8_desc(n, s, c_in, c_out, layout, dtype, training)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(s=-1), -1), (dict(c_in=0), -1), (dict(c_out=0), -1), (dict(layout=2), -1),
    (dict(layout=-1), -1), (dict(training=2), -1), (dict(dtype=2), -6), (dict(dtype=-1), -6),
    (dict(n=1 << 16, s=1 << 15), -10), (dict(c_in=(1 << 20) + 1), -10), (dict(c_out=(1 << 20) + 1), -10),
    (dict(n=1, s=0x7fffffff - 127), -10), (dict(n=1, s=1 << 27, c_in=1 << 12), -10),
    (dict(), 0), (dict(n=0), 0), (dict(s=0), 0), (dict(c_in=1 << 20, c_out=1), 0), (dict(training=0), 0),
    (dict(n=1, s=1 << 27, c_in=128, c_out=128), 0)])
def test_descriptor_refusals(kw, code):
    lib, d = L.load(), desc(**kw)
    ref = ctypes.byref(d)
    assert lib.deft_pw8_desc_validate(ref) == code
    if code:
        assert lib.deft_pw8_packed_bytes(ref) == lib.deft_pw8_saved_bytes(ref) == lib.deft_pw8_workspace_bytes(ref) == 0
        assert lib.deft_pw8_pack(ref, None, None, None) == code
        assert lib.deft_pw8_forward(ref, *[None] * 6, 0, None) == code
        assert lib.deft_pw8_backward(ref, *[None] * 7, 0, None) == code


def test_null_descriptor_and_empty_calls():
    lib = L.load()
    assert lib.deft_pw8_desc_validate(None) == -4
    assert lib.deft_pw8_packed_bytes(None) == lib.deft_pw8_saved_bytes(None) == lib.deft_pw8_workspace_bytes(None) == 0
    assert lib.deft_pw8_pack(None, None, None, None) == -4
    assert lib.deft_pw8_forward(None, *[None] * 6, 0, None) == -4
    assert lib.deft_pw8_backward(None, *[None] * 7, 0, None) == -4
    for kw in (dict(n=0), dict(s=0)):
        d = desc(**kw)
        assert lib.deft_pw8_forward(ctypes.byref(d), *[None] * 6, 0, None) == 0
        assert lib.deft_pw8_backward(ctypes.byref(d), *[None] * 7, 0, None) == 0
    assert lib.deft_pw8_backward(ctypes.byref(desc(training=0)), *[None] * 7, 0, None) == -1


def test_sizes():
    lib = L.load()
    d, infer = desc(c_in=300, c_out=130), desc(c_in=300, c_out=130, training=0)
    rows = 3 * 130 * 128 + 3 * 144  # codes and scales by blocks of the depth
    assert rows <= lib.deft_pw8_packed_bytes(ctypes.byref(infer)) <= rows + 1024
    turned = 2 * 300 * 128 + 2 * 304
    assert rows + turned <= lib.deft_pw8_packed_bytes(ctypes.byref(d)) <= rows + turned + 2048
    assert 2 * 300 * 128 <= lib.deft_pw8_saved_bytes(ctypes.byref(d)) <= 2 * 300 * 128 + 2048
    assert lib.deft_pw8_saved_bytes(ctypes.byref(infer)) == 0
    # single rows make their codes where they use them
    assert lib.deft_pw8_workspace_bytes(ctypes.byref(desc(n=16, s=1, training=0))) == 0
    assert lib.deft_pw8_workspace_bytes(ctypes.byref(desc(n=17, s=1, training=0))) > 0


@pytest.mark.fake_pointers
@pytest.mark.parametrize("layout", [0, 1])
def test_pointer_refusals(layout):
    lib, d = L.load(), desc(layout=layout)
    ref, far = ctypes.byref(d), 1 << 30
    ws = lib.deft_pw8_workspace_bytes(ref)
    pack = dict(w=FAKE, packed=far, stream=None)
    fwd = dict(x=FAKE, packed=FAKE, bias=FAKE, y=far, saved=2 * far, ws=FAKE, bytes=ws, stream=None)
    bwd = dict(saved=FAKE, packed=FAKE, dy=FAKE, dx=far, dw=far, db=far, ws=FAKE, bytes=ws, stream=None)

    def call(fn, base, **kw):
        return fn(ref, *{**base, **kw}.values())

    for fn, base, needed in ((lib.deft_pw8_pack, pack, ("w", "packed")),
                             (lib.deft_pw8_forward, fwd, ("x", "packed", "y", "saved")),
                             (lib.deft_pw8_backward, bwd, ("saved", "packed", "dy"))):
        for k in needed:
            assert call(fn, base, **{k: None}) == -4, k
        for k in [k for k in base if k not in ("ws", "bytes", "stream")]:
            assert call(fn, base, **{k: base[k] + 8}) == -7, k
        if "ws" in base:
            assert call(fn, base, ws=None) == -5
            assert call(fn, base, ws=FAKE + 4) == -7
    need = 2 * 100 * 128 + 208  # codes of x
    assert call(lib.deft_pw8_forward, fwd, bytes=need - 1) == -5
    assert call(lib.deft_pw8_backward, bwd, bytes=need - 1) == -5
    assert call(lib.deft_pw8_forward, fwd, y=FAKE) == -1
    assert call(lib.deft_pw8_forward, fwd, y=FAKE + 2 * 100 * 32 * 2 - 16) == -1
    assert call(lib.deft_pw8_backward, bwd, dx=FAKE) == -1
    assert call(lib.deft_pw8_pack, pack, packed=FAKE + 16) == -1


def test_python_class_refuses():
    for kw in (dict(layout="nchw"), dict(dtype="f16")):
        with pytest.raises(ValueError):
            Pointwise8(1, 8, 4, 8, device="cpu", **kw)
    with pytest.raises(L.DeftError):
        Pointwise8(1, 0, 4, 8, device="cpu")
    h = Pointwise8(2, 8, 20, 12, layout="channels_last", dtype="f32", training=True, device="cpu")
    x, w, b = torch.zeros(2, 20, 8), torch.zeros(12, 8), torch.zeros(12)
    packed, saved = torch.zeros(h.packed_bytes, dtype=torch.uint8), torch.zeros(h.saved_bytes, dtype=torch.uint8)
    dy = torch.zeros(2, 20, 12)
    for bad in (torch.zeros(12, 9), w.bfloat16(), torch.zeros(8, 12).t()):
        with pytest.raises(ValueError):
            h.pack(bad)
    with pytest.raises(ValueError):
        h.pack(w, out=packed[:-1])
    for bad in (dict(x=x[:1]), dict(x=x.double()), dict(x=x.transpose(0, 1)), dict(weights=w), dict(b=torch.zeros(8)),
                dict(y=x), dict(saved=packed)):
        with pytest.raises(ValueError):
            h.forward(**{**dict(x=x, weights=packed, b=b), **bad})
    for bad in (dict(saved=packed), dict(weights=saved), dict(dy=x), dict(out=dict(dz=x)), dict(out=dict(dx=dy))):
        with pytest.raises(ValueError):
            h.backward(**{**dict(saved=saved, weights=packed, dy=dy), **bad})
    with pytest.raises(ValueError):  # no GPU
        h.forward(x, packed, b)
    h = Pointwise8(2, 8, 20, 12, layout="channels_last", dtype="f32", device="cpu")
    with pytest.raises(ValueError):
        h.backward(saved, packed, dy)
    with pytest.raises(ValueError):
        h.forward(x, torch.zeros(h.packed_bytes, dtype=torch.uint8), b, saved=saved)


# ------------------------------------------------------------------ GPU

def rows_of(t, layout):
    """[rows][channels] of an image tensor."""
    return (t if layout == "channels_last" else t.transpose(1, 2)).reshape(-1, t.shape[2 if layout == "channels_last" else 1])


def image_of(rows, n, s, layout):
    t = rows.view(n, s, -1)
    return (t if layout == "channels_last" else t.transpose(1, 2)).contiguous()


def check(what, got, want, bound, dtype):
    off = (got.double() - want).abs()
    allowed = bound * (1 + HALF[dtype]) + want.abs() * HALF[dtype] + 2.0 ** -120
    bad = ~(off <= allowed) & ~(got.double() == want) & ~(torch.isnan(got) & torch.isnan(want))
    print("  %-3s worst error / bound %.3f" % (what, torch.nan_to_num(off / allowed).max().item()), flush=True)
    assert not bad.any(), (what, int(bad.sum()), off[bad][:4].tolist(), allowed[bad][:4].tolist())


def check_product(what, got, want, depth, dtype):
    want, mag, group, square = want
    steps = (-(-depth // 16) + min(512, -(-depth // 128)) + 1) * 2.0 ** -23
    over = mag > 2.0 ** 127  # not compared; NaN is
    got, want, mag, group = (torch.where(over, torch.zeros_like(t), t) for t in (got, want, mag, group))
    check(what, got, want, mag * steps + (group * 7 * 2.0 ** -13 if dtype == "bf16" else 0), dtype)
    if dtype == "bf16" and got.numel() >= 1000 and torch.isfinite(want).all():
        spread = 7 / 3 * 2.0 ** -26 * square + (want * HALF[dtype]).square() + (mag * steps).square()
        off = (got.double() - want).square().mean() / spread.mean()
        print("  %-3s spread / bound %.3f" % (what, off.sqrt().item()), flush=True)
        assert off <= 1, what


def inputs(n, c_in, s, c_out, layout, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def image(c):
        return image_of(rand(n * s, c) * torch.exp(rand(c)), n, s, layout).to(TYPES[dtype])

    return image(c_in), (rand(c_out, c_in) * torch.exp(rand(c_out, 1))).to(TYPES[dtype]), rand(c_out).to(TYPES[dtype]), image(c_out)


def run_and_check(n, c_in, s, c_out, layout, dtype, training=True, tensors=None):
    print("pw8", n, c_in, s, c_out, layout, dtype, training, flush=True)
    x, w, b, dy = tensors or inputs(n, c_in, s, c_out, layout, dtype)
    h = Pointwise8(n, c_in, s, c_out, layout=layout, dtype=dtype, training=training)
    packed = h.pack(w)
    y, saved = h.forward(x, packed, b)
    assert y.shape == ((n, s, c_out) if layout == "channels_last" else (n, c_out, s)) and y.dtype == TYPES[dtype]
    xr, dyr = rows_of(x, layout), rows_of(dy, layout)
    check_product("y", rows_of(y, layout), O.forward(xr, w, b), c_in, dtype)
    if not training:
        assert saved is None
        return
    g = h.backward(saved, packed, dy)
    want = O.backward(xr, w, dyr)
    check_product("dx", rows_of(g["dx"], layout), want["dx"], c_out, dtype)
    check_product("dw", g["dw"], want["dw"], n * s, dtype)
    check("db", g["db"], want["db"][0], want["db"][1] * 17 * 2.0 ** -24, dtype)


SHAPES = [  # n, c_in, s, c_out
    (1, 1, 1, 1), (1, 256, 1, 256), (16, 130, 1, 5), (17, 130, 1, 5), (1, 127, 129, 1), (3, 1, 50, 300), (2, 128, 64, 128),
    (5, 33, 7, 65), (40, 70, 3, 90), (1, 600, 130, 257), (3, 200, 333, 130), (2, 512, 1000, 384), (300, 40, 1, 24)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,c_in,s,c_out", SHAPES)
def test_matches_the_oracle(n, c_in, s, c_out, layout, dtype):
    run_and_check(n, c_in, s, c_out, layout, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,c_in,s,c_out", [(1, 1, 1, 1), (1, 8192, 1, 100), (3, 1000, 5, 33), (16, 128, 1, 9000),
                                            (2, 131, 8, 40), (4, 4100, 4, 17)])
def test_few_rows_match_the_oracle(n, c_in, s, c_out, layout, dtype):
    run_and_check(n, c_in, s, c_out, layout, dtype, training=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,c_in,s,c_out", [(8, 1024, 512, 4200), (1, 2048, 4097, 4225), (1, 520, 8300, 2050)])
def test_large_tiles_match_the_oracle(n, c_in, s, c_out, layout, dtype):
    run_and_check(n, c_in, s, c_out, layout, dtype)
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_few_rows_have_the_codes_of_the_other_calls(layout, dtype):
    """The same rows through the launch for few rows and among many: the sums' order may differ, the codes
    not, so with one block of channels and one-hot weights outputs are equal."""
    n, c, s = 4, 128, 4
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randn((n, c, s) if layout == "channels_first" else (n, s, c), generator=gen, device="cuda")
         * torch.exp(3 * torch.randn((n, 1, 1), generator=gen, device="cuda"))).to(TYPES[dtype])
    w = torch.eye(c, device="cuda", dtype=TYPES[dtype])
    h = Pointwise8(n, c, s, c, layout=layout, dtype=dtype)
    few, _ = h.forward(x, h.pack(w))
    big = Pointwise8(2 * n, c, s, c, layout=layout, dtype=dtype)
    many, _ = big.forward(torch.cat([x, x]), big.pack(w))
    assert torch.equal(few, many[:n]) and torch.equal(few, many[n:])
    want = image_of(O.coded(rows_of(x, layout)), n, s, layout)
    assert torch.equal(few.double(), want.to(TYPES[dtype]).double())


@pytest.mark.gpu
@pytest.mark.parametrize("training", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_values_that_are_not_finite_or_extreme(layout, training):
    n, c_in, s, c_out = (3, 260, 5, 140)
    x, w, b, dy = inputs(n, c_in, s, c_out, layout, "f32", seed=4)
    xr = rows_of(x, layout).clone()
    xr[2, 3], xr[4, 200], xr[7, 0] = float("inf"), float("nan"), -float("inf")
    xr[8], xr[9, :128], xr[10] = 0.0, 3e38, 1e-42
    xr[11, ::2] = 2.0 ** -127
    w[5, 9], w[139, 259] = float("nan"), float("inf")
    dyr = rows_of(dy, layout).clone()
    dyr[1, 2], dyr[14, 139] = float("nan"), -float("inf")
    run_and_check(n, c_in, s, c_out, layout, "f32", training,
                  (image_of(xr, n, s, layout), w, b, image_of(dyr, n, s, layout)))


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_no_bias_no_rows_and_chosen_gradients(layout):
    n, c_in, s, c_out = 3, 70, 60, 90
    x, w, b, dy = inputs(n, c_in, s, c_out, layout, "bf16", seed=5)
    h = Pointwise8(n, c_in, s, c_out, layout=layout, training=True)
    packed = h.pack(w)
    y, saved = h.forward(x, packed)
    check_product("y", rows_of(y, layout), O.forward(rows_of(x, layout), w), c_in, "bf16")
    full = h.backward(saved, packed, dy)
    for names in (["dx"], ["dw"], ["db"], ["dw", "db"], []):
        out = {k: torch.full_like(full[k], 7) for k in names}
        assert h.backward(saved, packed, dy, out=dict(out)).keys() == out.keys()
        got = h.backward(saved, packed, dy, out=out)
        for k in names:
            assert torch.equal(got[k], full[k]), k
    h = Pointwise8(0, c_in, s, c_out, layout=layout, training=True)
    empty, gone = x[:0], dy[:0]
    y, saved = h.forward(empty, packed, b)
    assert y.numel() == 0
    out = dict(dw=torch.full_like(w, 7), db=torch.full_like(b, 7))
    h.backward(saved, packed, gone, out=out)
    assert not out["dw"].any() and not out["db"].any()


@pytest.mark.gpu
def test_memory_behind_the_outputs_stays():
    n, c_in, s, c_out = 3, 130, 41, 77
    for layout in LAYOUTS:
        for dtype in ("f32", "bf16"):
            x, w, b, dy = inputs(n, c_in, s, c_out, layout, dtype, seed=6)
            h = Pointwise8(n, c_in, s, c_out, layout=layout, dtype=dtype, training=True)
            packed = h.pack(w)

            def guarded(count, t=TYPES[dtype]):
                return torch.full((count + 64,), 7, dtype=t, device="cuda")

            y, saved = guarded(n * s * c_out), guarded(h.saved_bytes, torch.uint8)
            h.forward(x, packed, b, y=y[:-64], saved=saved[:-64])
            out = dict(dx=guarded(n * s * c_in), dw=guarded(c_in * c_out), db=guarded(c_out))
            h.backward(saved[:-64], packed, dy, out={k: v[:-64] for k, v in out.items()})
            for t in (y, saved, *out.values()):
                assert (t[-64:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("training", [False, True])
@pytest.mark.parametrize("n,s", [(1, 9), (3, 200)])
def test_captured_calls_replay_like_eager_ones(n, s, training):
    c_in, c_out = 384, 130
    x, w, b, dy = inputs(n, c_in, s, c_out, "channels_last", "bf16", seed=7)
    h = Pointwise8(n, c_in, s, c_out, layout="channels_last", training=training)

    def step():
        packed = h.pack(w)
        y, saved = h.forward(x, packed, b)
        return [y] + (list(h.backward(saved, packed, dy).values()) if training else [])

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            held = step()
    for k in range(3):
        x.copy_(torch.roll(x, k + 1, 0) * (k + 1))
        w.mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(held, step()):
            assert torch.equal(got, want)
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_runs_on_the_current_stream():
    n, c_in, s, c_out = 2, 256, 500, 256
    x, w, b, dy = inputs(n, c_in, s, c_out, "channels_last", "bf16", seed=8)
    h = Pointwise8(n, c_in, s, c_out, layout="channels_last", training=True)
    packed = h.pack(w)
    want, saved = h.forward(x, packed, b)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = torch.zeros_like(x)
    with torch.cuda.stream(other):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
        y, again = h.forward(late, packed, b)
    other.synchronize()
    assert torch.equal(y, want) and torch.equal(again[:saved.numel() // 2], saved[:saved.numel() // 2])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_more_than_2_31_elements(layout):
    """x of 2^31 + 2^25 elements; rows at its start, in its middle and at its end against the oracle."""
    c_in, c_out, s = 8192, 40, (1 << 18) + 4099
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GiB of free memory")
    print("pw8", c_in, s, c_out, layout, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(71)
    shape = (1, s, c_in) if layout == "channels_last" else (1, c_in, s)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.randn((c_out, c_in), generator=gen, device="cuda").bfloat16()
    dy = torch.randn((1, s, c_out) if layout == "channels_last" else (1, c_out, s), generator=gen, device="cuda").bfloat16()
    h = Pointwise8(1, c_in, s, c_out, layout=layout, training=True)
    packed = h.pack(w)
    y, saved = h.forward(x, packed)
    g = h.backward(saved, packed, dy)

    def rows(t, at):
        return (t[0, at:at + 100] if layout == "channels_last" else t[0, :, at:at + 100].t()).contiguous()

    for at in (0, 1 << 17, (1 << 18) - 50, s - 100):
        check_product("y", rows(y, at), O.forward(rows(x, at), w), c_in, "bf16")
        want = O.backward(rows(x, at), w, rows(dy, at))["dx"]
        check_product("dx", rows(g["dx"], at), want, c_out, "bf16")
    # dw of the first and last channels
    xr = x[0] if layout == "channels_last" else x[0].t()
    dyr = dy[0] if layout == "channels_last" else dy[0].t()
    for part in (slice(0, 20), slice(c_in - 20, c_in)):
        want = O.product(O.coded(dyr.t()), O.coded(xr[:, part].t()).t())
        check_product("dw", g["dw"][:, part], want, s, "bf16")
    del x, y, saved, g
    torch.cuda.empty_cache()
