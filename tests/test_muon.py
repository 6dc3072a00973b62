"""Muon (deft_muon_step, optim.Muon).

CPU: the oracle, and every refusal of the C ABI and of the Python class.  GPU:
the direction against the oracle in float64, momentum and weights bit for bit.

Bounds of the direction, in Frobenius norms.  A step X -> A X + B X X^T X + ...
takes an error e of its X to at most STEEPEST |e|.  In each step and at its start
the kernels round: X and its three factors to 22 bits (2^-22 of each, by at most
a = 3.44, b and c of the step), their sums in fp32, whose roundings 2^-24 of
partial sums add up like a random walk of depth / 16 steps; and G, where a step
goes without X, by as much again.  32 * 2^-22 |X_k| for each step counts 8 such
roundings of at most 4 times the size of X each.  In one fp16 instead of a pair a
single rounding of X is 2^-11, 64 times that.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from irregular_gather_cnn_amd import _lib as L
from irregular_gather_cnn_amd.optim import ADJUST, AdamW, GradNorm, Muon
from oracle import muon as O

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ CPU: oracle

def test_oracle_acts_on_singular_values():
    r = np.random.default_rng(0)
    left, _ = np.linalg.qr(r.standard_normal((6, 6)))
    right, _ = np.linalg.qr(r.standard_normal((9, 6)))
    sigma = np.array([1.0, 0.6, 0.3, 0.05, 1e-3, 0.0])
    u = torch.from_numpy((left * sigma) @ right.T) * 7
    s = sigma / np.linalg.norm(sigma)
    for _ in range(5):
        s = O.A * s + O.B * s ** 3 + O.C * s ** 5
    for m in (u, u.t().contiguous()):
        x, _ = O.orthogonal(m, 5)
        want = (left * s) @ right.T
        np.testing.assert_allclose(x.numpy(), want if m is u else want.T, atol=1e-13)
    assert np.all((s[:4] > 0.6) & (s[:4] < 1.21)) and s[5] == 0


def test_oracle_of_tiny_and_zero_directions():
    assert not O.orthogonal(torch.zeros(3, 4), 5)[0].any()
    x, _ = O.orthogonal(torch.full((2, 2), 1e-12), 1, eps=1e-7)
    np.testing.assert_allclose(x.numpy(), O.A * 1e-5, rtol=1e-6)


def test_steepest_bounds_the_slope():
    s = torch.linspace(-1.21, 1.21, 100001, dtype=torch.float64)
    assert (O.A + 3 * O.B * s ** 2 + 5 * O.C * s ** 4).abs().max() <= O.STEEPEST + 1e-12
    p = O.A * s + O.B * s ** 3 + O.C * s ** 5
    assert p[s.abs() <= 1.21].abs().max() <= 1.21  # the range maps into itself


# ------------------------------------------------------------------ CPU: refusals

FAKE = 0x10000


def step_call(count=1, control=None, schedule=None, ws=FAKE, ws_bytes=1 << 40, desc=None, null=(), **tensor):
    d = dict(p_dtype=0, g_dtype=0, master=0, nesterov=1, steps=5, lr=0.02, momentum=0.95, eps=1e-7)
    t = dict(p=FAKE, g=FAKE, m=FAKE, master=None, rows=80, cols=240, weight_decay=0.0, scale=1.0)
    d.update(desc or {})
    t.update(tensor)
    d, t = L.deft_muon_desc(**d), (L.deft_muon_tensor * 1)(L.deft_muon_tensor(**t))
    return L.load().deft_muon_step(None if "desc" in null else ctypes.byref(d), None if "list" in null else t, count,
                                   control, schedule, ws, ws_bytes, None)


@pytest.mark.fake_pointers
@pytest.mark.parametrize("kw,code", [
    (dict(null=("desc",)), -4), (dict(null=("list",)), -4), (dict(p=None), -4), (dict(g=None), -4), (dict(m=None), -4),
    (dict(desc=dict(master=1, p_dtype=1)), -4), (dict(desc=dict(p_dtype=2)), -6), (dict(desc=dict(g_dtype=-1)), -6),
    (dict(count=-1), -1), (dict(rows=-1), -1), (dict(cols=-1), -1), (dict(weight_decay=-0.1), -1),
    (dict(weight_decay=math.nan), -1), (dict(scale=math.inf), -1), (dict(scale=math.nan), -1),
    (dict(desc=dict(master=1)), -1), (dict(desc=dict(master=2, p_dtype=1)), -1), (dict(desc=dict(steps=0)), -1),
    (dict(desc=dict(steps=33)), -1), (dict(desc=dict(nesterov=2)), -1), (dict(desc=dict(lr=-1.0)), -1),
    (dict(desc=dict(lr=math.inf)), -1), (dict(desc=dict(momentum=1.0)), -1), (dict(desc=dict(momentum=math.nan)), -1),
    (dict(desc=dict(momentum=-0.1)), -1), (dict(desc=dict(eps=0.0)), -1), (dict(desc=dict(eps=math.nan)), -1),
    (dict(p=FAKE + 4), -7), (dict(g=FAKE + 8), -7), (dict(m=FAKE + 4), -7),
    (dict(master=FAKE + 4, desc=dict(master=1, p_dtype=1)), -7), (dict(control=FAKE + 2), -7),
    (dict(schedule=FAKE + 4), -7), (dict(ws=FAKE + 4), -7), (dict(ws=None), -5), (dict(ws_bytes=100), -5),
    (dict(rows=(1 << 15) + 1, cols=(1 << 15) + 1), -10), (dict(rows=1, cols=(1 << 22) + 1), -10),
    (dict(rows=1 << 11, cols=(1 << 21) + 1), -10)])
def test_refuses(kw, code):
    assert step_call(**kw) == code


def test_empty_lists_are_no_ops():
    assert step_call(count=0, null=("list",)) == 0
    assert step_call(rows=0, p=None, g=None, m=None, ws=None, ws_bytes=0) == 0
    assert step_call(cols=0, p=None, g=None, m=None, ws=None, ws_bytes=0) == 0


def test_workspace_bytes():
    lib = L.load()

    def need(*shapes):
        t = (L.deft_muon_tensor * len(shapes))(*[L.deft_muon_tensor(rows=r, cols=c) for r, c in shapes])
        return lib.deft_muon_workspace_bytes(t, len(shapes))

    assert lib.deft_muon_workspace_bytes(None, 0) == need((0, 5)) == need((5, 0)) == 0
    assert need((-1, 5)) == need((1, (1 << 22) + 1)) == 0
    # two copies of X and six squares, each of 4 bytes an element, at least
    assert need((256, 2304)) >= 4 * (2 * 256 * 2304 + 6 * 256 * 256)
    assert need((256, 2304)) == need((2304, 256))
    # a long list reuses what a launch's matrices need
    assert need(*[(65, 65)] * 96) == need(*[(65, 65)] * 48) > 0
    # matrices that fit one workgroup's memory need none, where all do
    assert need((64, 64), (18, 144), (900, 3)) == 0 and need((64, 64), (65, 65)) > 0 and need((2, 2000)) > 0


def test_python_class_refuses():
    def make(shapes=((4, 6), (3, 2, 5)), dtype=torch.bfloat16, **kw):
        p = [torch.zeros(s, dtype=dtype) for s in shapes]
        return p, [torch.zeros_like(t) for t in p], kw

    def muon(p, g, kw):
        return Muon(p, g, **kw)

    with pytest.raises(ValueError):
        Muon([], [])
    for bad in (dict(adjust="lr"), dict(masters=[torch.zeros(24)]), dict(states=[torch.zeros(24)]),
                dict(weight_decay=[0.1]), dict(states=[torch.zeros(24), torch.zeros(29)]),
                dict(states=[torch.zeros(24), torch.zeros(30, dtype=torch.float64)]),
                dict(masters=[torch.zeros(24), None])):
        with pytest.raises(ValueError):
            muon(*make(**bad))
    with pytest.raises(ValueError):
        muon(*make(shapes=((4, 6), (7,))))
    p, g, kw = make()
    with pytest.raises(ValueError):
        Muon([p[0], p[0]], [g[0], g[0]])
    for bad in (g[:1], [g[0], g[1][:2]], [g[0], torch.zeros(3, 2, 5)]):
        with pytest.raises((ValueError, TypeError)):
            Muon(p, bad)
    with pytest.raises(TypeError):
        Muon([p[0], torch.zeros(2, 2)], g)
    with pytest.raises(ValueError):
        Muon([p[0].t(), p[1]], g)
    opt = Muon(p, g)
    for bad in (dict(control=torch.zeros(3)), dict(control=torch.zeros(4, dtype=torch.float64)),
                dict(schedule=torch.zeros(1)), dict(schedule=torch.zeros(2, dtype=torch.float64))):
        with pytest.raises(ValueError):
            opt.step(**bad)
    with pytest.raises(ValueError):
        opt.bind(g[:1])
    with pytest.raises(ValueError):  # no GPU
        opt.step()


def test_handles_hold_the_memory_they_point_to():
    p, g = ([torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 6), (3, 2, 5))] for _ in range(2))
    opt = Muon(p, g, masters=True)
    for t in p + g + opt.masters + opt.states:
        t.data = torch.empty_like(t)
    kept = {t.data_ptr() for t in opt._held + opt.grads.held}
    for item in opt._list:
        for field in ("p", "g", "m", "master"):
            assert getattr(item, field) in kept, field


def test_adjust():
    assert ADJUST["none"](9, 4) == 1.0 and ADJUST["aspect"](9, 4) == 1.5 and ADJUST["aspect"](4, 9) == 1.0
    assert abs(ADJUST["rms"](9, 4) - 0.6) < 1e-15


# ------------------------------------------------------------------ GPU

def rand(shape, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda") * scale


def direction(us, steps=5, eps=1e-7):
    """X of each u: a step from zero weights with no momentum, whose new weights are -X."""
    p = [torch.zeros_like(u) for u in us]
    opt = Muon(p, us, lr=1.0, momentum=0.0, nesterov=False, weight_decay=0.0, steps=steps, adjust="none", eps=eps)
    opt.step()
    for m, u in zip(opt.states, us):
        assert torch.equal(m.view_as(u), u)
    return [-q for q in p]


def check_direction(us, steps=5, eps=1e-7):
    print("muon", [tuple(u.shape) for u in us[:8]], steps, flush=True)
    for u, x in zip(us, direction(us, steps, eps)):
        want, sizes = O.orthogonal(u.view(u.shape[0], -1), steps, eps)
        off = float(torch.linalg.vector_norm(x.view_as(want).double() - want))
        bound = 32 * 2.0 ** -22 * sizes
        print("  %s off %.2e of %.2e, bound %.2e" % (tuple(u.shape), off, float(want.norm()), bound), flush=True)
        assert off <= bound


LARGE = (70, 90)  # with it in a list, no matrix takes the launch for small ones
SHAPES = [(1, 1), (1, 7), (9, 1), (5, 3), (16, 144), (18, 144), (31, 33), (64, 64), (65, 32), (130, 70), (128, 129), (300, 1000),
          (1000, 300), (18, 2304), (256, 2304), (513, 513), (33, 5000)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
def test_direction_matches_the_oracle(shape):
    check_direction([rand(shape, 1)])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [s for s in SHAPES if min(s) <= 64] + [(32, 960), (960, 32), (64, 352), (352, 64), (33, 31)])
def test_small_matrices_among_large_ones(shape):
    check_direction([rand(shape, 1), rand(LARGE, 2), rand(shape, 3)])
    check_direction([rand(shape, 4), rand(shape, 5)])


@pytest.mark.gpu
@pytest.mark.parametrize("shapes", [[(1024, 1100), (600, 2300), (1500, 700)], [(2100, 2049)], [(300, 5000)] * 9,
                                    [(40, 60000), (60000, 33)], [(6000, 6100)], [(1100, 9000), (9000, 1100)]])
def test_large_tiles(shapes):
    check_direction([rand(s, 6 + k) for k, s in enumerate(shapes)])
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 7, 10, 32])
def test_any_number_of_steps(steps):
    # from 6 steps on an error's part that grows in all of them leaves the bound no meaning: the steps come to
    # rest between 0.68 and 1.21, which is checked instead
    us = [rand((40, 100), 2), rand((130, 70), 3)]
    if steps < 6:
        check_direction(us[:1], steps)
        return check_direction(us, steps)
    for u, x in zip(us, direction(us, steps)):
        s = torch.linalg.svdvals(x.double().cpu())
        assert s.min() > 0.65 and s.max() < 1.22
        c = x.double() @ u.double().t()  # X U^T is symmetric with positive eigenvalues, as X's singular vectors are U's
        assert float((c - c.t()).norm() / c.norm()) < 1e-3


def spectra(m, n):
    """Normal values; few strong directions in noise; singular values over five decades; one direction."""
    k = max(1, m // 8)
    q1 = torch.linalg.qr(rand((m, m), 5).double().cpu())[0]
    q2 = torch.linalg.qr(rand((n, m), 6).double().cpu())[0]
    return dict(normal=rand((m, n), 4), strong=rand((m, k), 7) @ rand((k, n), 8) + 0.02 * rand((m, n), 9),
                decades=((q1 * torch.logspace(0, -5, m, dtype=torch.float64)) @ q2.t()).float().cuda(),
                one=rand((m, 1), 10) @ rand((1, n), 11))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["normal", "strong", "decades", "one"])
@pytest.mark.parametrize("m,n", [(64, 64), (64, 300), (256, 700), (200, 200)])
def test_directions_are_as_near_as_steps_in_fp32(m, n, name):
    """Each step's products in fp32 torch, on the CPU, are the measure: no more than 4 times as far."""
    u = spectra(m, n)[name]
    x = (u / torch.linalg.vector_norm(u.double()).float()).cpu()
    for _ in range(5):
        g = x @ x.t()
        x = O.A * x + (O.B * g + O.C * (g @ g)) @ x
    want, sizes = O.orthogonal(u, 5)
    plain = float((x.double() - want.cpu()).norm())
    for v in (u, u.t().contiguous()):
        got = direction([v])[0]
        off = float(((got if v is u else got.t()).double() - want).norm())
        print("muon %s %dx%d off %.2e, fp32 steps %.2e, bound %.2e" % (name, m, n, off, plain, 32 * 2.0 ** -22 * sizes),
              flush=True)
        assert off <= 4 * plain + 2.0 ** -22 * float(want.norm())


@pytest.mark.gpu
def test_sizes_of_directions():
    """The direction does not depend on the gradient's size down to eps, below it shrinks; zero stays zero."""
    u = rand((40, 90), 12)
    base = direction([u])[0].double()
    for scale in (2.0 ** 60, 2.0 ** -40, 2.0 ** -20):
        assert torch.equal(direction([u * scale], eps=1e-30)[0].double(), base)
    check_direction([u * 1e-9, u * 1e-12])
    assert not direction([torch.zeros_like(u)])[0].any()
    check_direction([u * 1e30, u * 1e-25], eps=1e-30)


@pytest.mark.gpu
def test_a_matrix_that_is_not_finite_stays_alone():
    for extra in ([], [rand(LARGE, 16)]):
        us = [rand((40, 90), 13), rand((100, 30), 14), rand((7, 7), 15)] + extra
        want = direction(us)
        for bad in (math.nan, math.inf, -math.inf):
            us[1][50, 3] = bad
            got = direction_with_states(us)
            assert torch.isnan(got[1]).all()
            assert all(torch.equal(got[k], want[k]) for k in range(len(us)) if k != 1)


def direction_with_states(us):
    p = [torch.zeros_like(u) for u in us]
    Muon(p, us, lr=1.0, momentum=0.0, nesterov=False, weight_decay=0.0, adjust="none").step()
    return [-q for q in p]


def training(p_type, g_type, master, shapes, seed=20):
    p = [rand(s, seed + k, 0.05) for k, s in enumerate(shapes)]
    masters = [q.clone() for q in p] if master else None
    p = [q.to(TYPES[p_type]) for q in p]
    g = [rand(s, seed + 50 + k, 1e-3).to(TYPES[g_type]) for k, s in enumerate(shapes)]
    m = [rand(s, seed + 90 + k, 1e-3) for k, s in enumerate(shapes)]
    return p, g, m, masters


@pytest.mark.gpu
@pytest.mark.parametrize("small", [True, False])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("clip", [True, False])
@pytest.mark.parametrize("p_type,g_type,master", [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", False),
                                                  ("bf16", "bf16", True), ("bf16", "f32", True)])
def test_momentum_and_weights_bit_for_bit(p_type, g_type, master, clip, nesterov, small):
    """The direction of a step from zero weights gives the same bits, so the weights are compared with the
    formula on it."""
    shapes = [(16, 4, 3, 3), (90, 30), (33, 70), (5, 5), (2, 200 if small else 2000)]
    p, g, m, masters = training(p_type, g_type, master, shapes)
    decay = [0.0, 0.1, 0.01, 0.3, 0.0]
    print("muon", p_type, g_type, master, clip, nesterov, flush=True)
    before = [t.clone() for t in p], [t.clone() for t in m], [t.clone() for t in masters or []]
    hyper = dict(momentum=0.9, nesterov=nesterov, adjust="rms")
    opt = Muon(p, g, lr=0.03, weight_decay=decay, masters=masters, states=m, **hyper)
    zero = [torch.zeros(s, device="cuda") for s in shapes]
    probe = Muon(zero, g, lr=1.0, weight_decay=0.0, states=[t.clone() for t in m], **{**hyper, "adjust": "none"})
    control = opt.grad_norm(max_norm=0.01) if clip else None
    opt.step(control=control)
    probe.step(control=control)
    for k, s in enumerate(shapes):
        rows, cols = s[0], math.prod(s[1:])
        mom, u = O.momentum(before[1][k], g[k], 0.9, nesterov, control[1] if clip else None)
        assert torch.equal(m[k], mom) and torch.equal(probe.states[k], mom)
        x, sizes = O.orthogonal(u.view(rows, cols), 5)
        assert float((-zero[k].view(rows, cols).double() - x).norm()) <= 32 * 2.0 ** -22 * sizes
        full = O.update(before[2][k] if master else before[0][k], -zero[k], 0.03, decay[k], 0.2 * math.sqrt(max(rows, cols)))
        if master:
            assert torch.equal(masters[k], full)
        assert torch.equal(p[k], full.to(p[k].dtype))


@pytest.mark.gpu
def test_long_lists_take_several_launches():
    shapes = [(8 + k % 5, 9 + k) for k in range(101)] + [(0, 4), (60, 0), (70, 3)]
    us = [rand(s, 200 + k) for k, s in enumerate(shapes)]
    got = direction(us)
    for k in (0, 46, 47, 48, 49, 95, 96, 97, 100, 103):
        assert torch.equal(got[k], direction([us[k]])[0])
    check_direction(us[:101:10] + us[103:])
    us[60] = rand(LARGE, 500)  # the second launch's matrices are not all small, then
    check_direction(us[:101] + us[103:])


@pytest.mark.gpu
@pytest.mark.parametrize("small", [True, False])
def test_gradients_that_are_not_finite_skip_the_step(small):
    p, g, m, masters = training("bf16", "bf16", True, [(40, 50), (200, 20)] + ([] if small else [LARGE]))
    opt = Muon(p, g, masters=masters, states=m)
    before = [t.clone() for t in p + m + masters]
    g[1][3, 3] = math.inf
    control = opt.grad_norm(max_norm=1.0)
    opt.step(control=control)
    assert control[2] == 0 and all(torch.equal(a, b) for a, b in zip(before, p + m + masters))
    g[1][3, 3] = 0.5
    opt.step(control=opt.grad_norm(max_norm=1.0))
    assert all(not torch.equal(a, b) and torch.isfinite(b).all() for a, b in zip(before, p + m + masters))


@pytest.mark.gpu
def test_one_norm_clips_matrices_and_vectors():
    """One GradNorm over all gradients, for Muon's matrices and AdamW's vectors."""
    w, gw = [rand((30, 40), 1, 0.1)], [rand((30, 40), 2)]
    b, gb = [rand((30,), 3, 0.1)], [rand((30,), 4)]
    control = GradNorm(gw + gb)(max_norm=0.5)
    norm = math.sqrt(float(gw[0].double().square().sum() + gb[0].double().square().sum()))
    assert abs(control[1].item() * norm / 0.5 - 1) < 1e-5
    muon, adam = Muon(w, gw), AdamW(b, gb)
    muon.step(control=control)
    adam.step(control=control)
    want, _ = O.momentum(torch.zeros_like(w[0]), gw[0], 0.95, True, control[1])
    assert torch.equal(muon.states[0].view_as(want), want)


@pytest.mark.gpu
def test_schedule_on_the_device_and_lr():
    shapes = [(20, 30), (50, 20)]
    runs = []
    for form in ("host", "device", "both"):
        p, g, m, _ = training("f32", "f32", False, shapes)
        opt = Muon(p, g, lr=0.5 if form == "both" else 0.02, states=m)
        for lr in (0.02, 0.01, 0.003):
            schedule = torch.tensor([lr], dtype=torch.float64, device="cuda") if form != "host" else None
            opt.step(lr=lr if form == "host" else None, schedule=schedule)
        runs.append(p)
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


@pytest.mark.gpu
@pytest.mark.parametrize("shapes", [[(16, 4, 3, 3), (200, 90), (64, 1000)], [(16, 4, 3, 3), (5, 70)]])
def test_captured_step_replays_like_eager_steps(shapes):
    p, g, m, masters = training("bf16", "bf16", True, shapes)
    q = [[t.clone() for t in part] for part in (p, m, masters)]
    lr = torch.tensor([0.02], dtype=torch.float64, device="cuda")
    opt = Muon(p, g, masters=masters, states=m)
    eager = Muon(q[0], g, masters=q[2], states=q[1])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            opt.step(control=opt.grad_norm(max_norm=0.1), schedule=lr)
    for k in range(4):
        for t in g:
            t.copy_(torch.roll(t, k + 1, 0) * 1.5)
        lr.fill_(0.02 / (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        eager.step(control=eager.grad_norm(max_norm=0.1), lr=0.02 / (k + 1))
        for a, b in zip(p + m + masters, q[0] + q[1] + q[2]):
            assert torch.equal(a, b), k
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_runs_on_the_current_stream_and_on_rebound_gradients():
    p, g, m, _ = training("f32", "f32", False, [(40, 60), (100, 30)])
    q, n = [t.clone() for t in p], [t.clone() for t in m]
    opt, want = Muon(p, g, states=m), Muon(q, [t * 2 + 1e-4 for t in g], states=n)
    want.step()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    late = [torch.zeros_like(t) for t in g]
    opt.bind(late)
    with torch.cuda.stream(other):
        torch.cuda._sleep(20_000_000)
        for a, b in zip(late, g):
            a.copy_(b * 2 + 1e-4)
        opt.step()
    other.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(p + m, q + n))


@pytest.mark.gpu
@pytest.mark.parametrize("shapes", [[(17, 45), (45, 17), (130, 3)], [(17, 45), (45, 17), (130, 3), (67, 71)]])
def test_memory_behind_the_tensors_stays(shapes):
    flat = torch.full((4, 8192), 7.0, device="cuda")
    for dtype in TYPES.values():
        base, moms = flat.to(dtype, copy=True), flat.clone()
        p = [base[k, :r * c].view(r, c) for k, (r, c) in enumerate(shapes)]
        m = [moms[k, :r * c] for k, (r, c) in enumerate(shapes)]
        # a bf16 weight of 7 moves by steps of 2^-5: lr 1 moves it
        opt = Muon(p, [rand(s, 60).to(dtype) for s in shapes], lr=1.0, states=m)
        opt.ws = torch.full((opt.ws_bytes + 1024,), 0x7e, dtype=torch.uint8, device="cuda")  # fp16 0x7e7e: NaN
        opt._ws = opt.ws.data_ptr()
        opt.step()
        for k, (r, c) in enumerate(shapes):
            assert (base[k, r * c:] == 7).all() and (moms[k, r * c:] == 7).all()
            assert torch.isfinite(p[k]).all() and not (p[k] == 7).all()
        assert (opt.ws[opt.ws_bytes:] == 0x7e).all()


@pytest.mark.gpu
def test_more_than_2_31_elements():
    """The direction is P X0 with P a polynomial of X0 X0^T, which is summed up here in float64 by pieces."""
    m, n = 520, (1 << 22) - 32
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GiB of free memory")
    print("muon", m, n, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(70)
    u = torch.randn((m, n), generator=gen, device="cuda")
    p = torch.zeros_like(u)
    opt = Muon([p], [u], lr=1.0, momentum=0.0, nesterov=False, weight_decay=0.0, adjust="none")
    opt.step()
    gram = torch.zeros((m, m), dtype=torch.float64, device="cuda")
    for j in range(0, n, 1 << 18):
        piece = u[:, j:j + (1 << 18)].double()
        gram += piece @ piece.t()
    norm = gram.diagonal().sum().sqrt()
    gram /= norm * norm
    poly, eye = torch.eye(m, dtype=torch.float64, device="cuda"), torch.eye(m, dtype=torch.float64, device="cuda")
    sizes = 0.0
    for _ in range(5):
        sizes = O.STEEPEST * (sizes + float(gram.diagonal().sum().sqrt()))
        q = O.A * eye + O.B * gram + O.C * gram @ gram
        poly, gram = q @ poly, q @ gram @ q
    bound = 32 * 2.0 ** -22 * (sizes + float(gram.diagonal().sum().sqrt()))
    for j in (0, 1 << 20, n - 5000):
        want = poly @ (u[:, j:j + 5000].double() / norm)
        off = (-p[:, j:j + 5000].double() - want).norm()
        # the columns are alike: an error's share of these is that of their number, 4 times that at most
        assert float(off) <= 4 * bound * math.sqrt(5000 / n), j
        assert float(want.norm()) > 100 * float(off)
    del u, p, opt
    torch.cuda.empty_cache()
