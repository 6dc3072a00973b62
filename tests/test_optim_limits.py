"""AdamW at the ends of its range: launches have fewer than 2^32 threads, of 1024 elements a 256; and the
memory that its handles point to."""
import gc

import pytest
import torch

from irregular_gather_cnn_amd.optim import AdamW, GradNorm
from test_optim import FAKE, step_call

MOST = (2 ** 24 - 1) * 1024  # elements of one launch


@pytest.mark.fake_pointers
@pytest.mark.parametrize("n,code", [(MOST, -4), (MOST + 1, -10)])
def test_a_tensor_of_more_than_one_launch_is_refused(n, code):
    """Before its pointers are looked at: the smaller one's missing weights are, then."""
    assert step_call(n=n, p=None, g=FAKE) == code


@pytest.mark.gpu
def test_a_list_of_more_than_one_launch():
    """Two tensors that one launch does not hold: every weight moves like that of a small tensor, as all
    gradients are alike."""
    sizes = [MOST - 1024, 4097]
    if torch.cuda.mem_get_info()[0] < 7 * sum(sizes):
        pytest.skip("needs 7 bytes of free memory an element, for 2^34 elements")
    print("adamw", sizes, flush=True)

    def run(sizes):
        p = [torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda") for n in sizes]
        opt = AdamW(p, [torch.full((n,), 1e-3, dtype=torch.bfloat16, device="cuda") for n in sizes], lr=1e-2, bits=8,
                    weight_decay=0.0)
        opt.step()
        return p

    want = run([5])[0][0]
    assert want != 0.5
    for t in run(sizes):
        assert t.min() == t.max() == want
    torch.cuda.empty_cache()


@pytest.mark.parametrize("bits", [8, 32])
def test_handles_hold_the_memory_they_point_to(bits):
    """Also where every tensor of the program gets other memory."""
    sizes = [300, 7]
    p, g = ([torch.zeros(n, dtype=torch.bfloat16) for n in sizes] for _ in range(2))
    opt, norm = AdamW(p, g, bits=bits, masters=True), GradNorm(g)
    for t in p + g + opt.masters + [t for s in opt.states for t in s if t is not None]:
        t.data = torch.empty_like(t)
    gc.collect()
    kept = {t.data_ptr() for t in opt._held + opt.grads.held + norm.grads.held}
    for item in opt._list:
        for field in ("p", "g", "m", "v", "master") + (("m_scale", "v_scale") if bits == 8 else ()):
            assert getattr(item, field) in kept, field
    assert set(norm.grads.pointers) <= kept
