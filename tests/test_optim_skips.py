"""Steps that control skips leave no mark on later ones: their bias corrections
count the steps that were taken.
"""
import numpy as np
import pytest
import torch

from irregular_gather_cnn_amd.optim import AdamW
from oracle import optim as O
from test_optim import HYPER, KINDS, Mirror, host, make, step_call

H = 2.0 ** -24


@pytest.mark.fake_pointers
def test_the_count_is_aligned():
    import ctypes

    from irregular_gather_cnn_amd import _lib as L
    d = L.deft_adamw_desc(0, 0, 32, 0, 1, 1e-3, 0.9, 0.999, 1e-8, 0, 0x10002)
    t = (L.deft_adamw_tensor * 1)()
    assert L.load().deft_adamw_step(ctypes.byref(d), t, 1, None, None, None) == -7
    assert step_call(count=0) == 0


def skip(opt, g):
    keep = g[0][0].item()
    g[0][0] = float("inf")
    opt.step(control=opt.grad_norm())
    g[0][0] = keep


@pytest.mark.gpu
@pytest.mark.parametrize("p_type,g_type,bits,master", KINDS)
def test_the_first_step_after_skipped_ones_is_a_first_step(p_type, g_type, bits, master):
    """m and v are those of a fresh run, bit for bit.  The factors of the update may differ by the rounding of
    the device's powers: each by one unit in fp32, and the update by two more roundings."""
    print("adamw", p_type, g_type, bits, master, flush=True)
    sizes = [5000, 18, 257]
    a, ga, _ = make(sizes, p_type, g_type, bits, master, 21)
    b, gb, _ = make(sizes, p_type, g_type, bits, master, 21)
    before = [host(t) for t in a.masters or a.params]
    for _ in range(4):
        skip(a, ga)
    a.step(control=a.grad_norm())
    b.step(control=b.grad_norm())
    assert a.steps == 5 and a.taken() == 1 and b.taken() == 1
    for k in range(len(sizes)):
        x, y = (host((o.masters or o.params)[k]).astype(np.float64) for o in (a, b))
        moved = np.abs(y - before[k]) + H * np.abs(y)
        half = 0 if master else {"f32": 0, "bf16": 2.0 ** -7}[p_type]  # either neighbour
        assert (np.abs(x - y) <= 8 * H * moved + 2 * H * np.abs(y) + half * np.abs(y)).all()
        assert not np.array_equal(x, before[k])
        # the seeds of the 8-bit roundings of sqrt(v) are those of steps 5 and 1
        for got, want in list(zip(a.states[k], b.states[k]))[0:4:2 if bits == 8 else 1]:
            if got is not None:
                np.testing.assert_array_equal(host(got), host(want))


@pytest.mark.gpu
def test_skips_between_steps_match_the_oracle_of_the_steps_taken():
    opt, g, decay = make([3000, 40], "f32", "f32", 32, False, 22)
    mir = Mirror(opt, decay)
    taken = 0
    for k in range(12):
        for t in g:
            t.mul_(-0.8)
        if k % 3 == 1:
            skip(opt, g)
            continue
        taken += 1
        mir.read()
        control = opt.grad_norm()
        opt.step(control=control)
        assert opt.taken() == taken
        for j in range(2):
            m, v = mir.state[j][:2]
            p64, m64, v64, root = O.adamw(mir.p[j], host(g[j]), m, v, step=taken, lr=HYPER["lr"], beta1=0.9,
                                          beta2=0.999, eps=1e-8, weight_decay=decay[j])
            # the bounds of test_steps_match_the_oracle, with one more rounding of either factor
            em = 6 * H * (0.9 * np.abs(m) + 0.1 * np.abs(host(g[j])))
            rate = HYPER["lr"] / (1 - 0.9 ** taken)
            den = root / np.sqrt(1 - 0.999 ** taken) + 1e-8
            ep = 3 * H * np.abs(mir.p[j]) + rate / den * (em + 18 * H * np.abs(m64)) + 1e-40
            assert (np.abs(host(opt.params[j]) - p64) <= ep).all()
            # a step's number too many would be seen
            late = O.adamw(mir.p[j], host(g[j]), m, v, step=k + 1, lr=HYPER["lr"], beta1=0.9, beta2=0.999, eps=1e-8,
                           weight_decay=decay[j])[0]
            assert k == 0 or (np.abs(late - p64) > 4 * ep).any()


@pytest.mark.gpu
def test_a_long_list_counts_a_skipped_step_once():
    opt, g, _ = make([100] * 120, "bf16", "bf16", 8, True, 23)
    for _ in range(3):
        skip(opt, g)
    assert opt.skipped.item() == 3
    opt.step(control=opt.grad_norm())
    assert opt.steps == 4 and opt.taken() == 1


@pytest.mark.gpu
def test_no_first_moment_has_no_correction():
    """beta1 = 0: 1 - 0^t is 1 for every t."""
    p, g = [torch.ones(300, device="cuda")], [torch.full((300,), 0.5, device="cuda")]
    opt = AdamW(p, g, lr=0.25, betas=(0.0, 0.999), eps=0.0, weight_decay=0.0)
    skip(opt, g)
    opt.step(control=opt.grad_norm())
    # the first step moves by lr, off by its roundings
    assert (p[0] - 0.75).abs().max() <= 16 * H


@pytest.mark.gpu
def test_a_captured_step_counts_its_skips_on_the_device():
    opt, g, _ = make([700], "f32", "f32", 32, False, 24)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(control=opt.grad_norm())
    before = [t.clone() for t in opt.params + [t for t in opt.states[0] if t is not None]]
    g[0][5] = float("nan")
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert opt.skipped.item() == k + 1
        for a, b in zip(opt.params + [t for t in opt.states[0] if t is not None], before):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_what_a_call_leaves_for_the_next_one_is_what_that_would_compute():
    """The corrections that the last call left, and those computed where it left none: the same bits."""
    a, ga, _ = make([3000, 40], "bf16", "bf16", 8, True, 25)
    b, gb, _ = make([3000, 40], "bf16", "bf16", 8, True, 25)
    for k in range(8):
        for opt, g in ((a, ga), (b, gb)):
            if opt is b:
                opt._skips[4:].zero_()
            if k in (1, 2, 5):
                skip(opt, g)
            else:
                opt.step(control=opt.grad_norm())
        for x, y in zip(a.params + a.masters + [t for s in a.states for t in s],
                        b.params + b.masters + [t for s in b.states for t in s]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert a.taken() == b.taken() == 5
