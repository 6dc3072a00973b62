"""Group norm where the mean dominates: the forward computes z from x - mean in
both types, as the backward does.
"""
import numpy as np
import pytest
import torch

from irregular_gather_cnn_amd.norm import GroupNormAct

pytestmark = pytest.mark.gpu
LAYOUTS = ["channels_first", "channels_last"]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# groups that one workgroup holds, that several share, and that are read twice
SIZES = [(2, 16, 60, 4), (2, 16, 30011, 4), (1, 48, 700003, 3)]


def fill(values, n, s, layout, dtype):
    """x [n][c][s], each channel one number, in the layout."""
    v = torch.tensor(values, dtype=TYPES[dtype], device="cuda")
    x = v.view(1, -1, 1).expand(n, len(values), s)
    return (x.transpose(1, 2) if layout == "channels_last" else x).contiguous()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("eps", [1e-5, 1e-6])
@pytest.mark.parametrize("size", SIZES, ids=lambda v: "x".join(map(str, v)))
def test_constant_groups_give_beta(size, eps, layout, dtype):
    """x equals its mean, which every sum holds exactly: z = beta, at any mean, and so y = act(beta)
    without a rounding; dx is what the gradients' own sums give at h = 0."""
    n, c, s, g = size
    print("norm", size, eps, layout, dtype, flush=True)
    beta = torch.linspace(-1, 1, c).to(TYPES[dtype]).cuda()
    gamma = torch.linspace(0.5, 1.5, c).to(TYPES[dtype]).cuda()
    for name in ("none", "relu"):
        h = GroupNormAct(n, c, s, g, eps=eps, act=name, layout=layout, dtype=dtype)
        want = beta.clamp(min=0) if name == "relu" else beta
        want = want.view((1, 1, c) if layout == "channels_last" else (1, c, 1))
        for level in (100.0, 1000.0, -1000.0, 29952.0):
            x = fill([level * 2.0 ** (k // (c // g)) for k in range(c)], n, s, layout, dtype)
            y, mean, rstd = h.forward(x, gamma, beta)
            assert torch.equal(mean, torch.tensor([level * 2.0 ** k for k in range(g)], device="cuda").expand(n, g))
            assert torch.equal(y, want.expand_as(y)), level


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("level", [0.0, 3.0, 100.0, 1000.0])
def test_relu_passes_the_same_elements_forward_and_backward(level, layout, dtype):
    """With dy = 1, dbeta counts the elements that the backward passes: as many as y shows above zero.
    128 positions, so that the counts are exact in bf16; constant groups and others."""
    n, c, s, g = 2, 32, 64, 4
    r = np.random.default_rng(3)
    v = level + r.standard_normal((n, c, s)) * 4 * (np.arange(c) % 16 >= 8)[None, :, None]  # groups 0 and 2 constant
    x = torch.from_numpy(v).to(TYPES[dtype])
    x = (x.transpose(1, 2) if layout == "channels_last" else x).contiguous().cuda()
    gamma = torch.from_numpy(r.standard_normal(c)).to(TYPES[dtype]).cuda()
    for beta in (torch.zeros_like(gamma), (gamma * 0.25).to(TYPES[dtype])):
        h = GroupNormAct(n, c, s, g, act="relu", layout=layout, dtype=dtype, training=True)
        y, mean, rstd = h.forward(x, gamma, beta)
        out = h.backward(x, gamma, beta, mean, rstd, torch.ones_like(x))
        shown = (y > 0).sum((0, 1) if layout == "channels_last" else (0, 2))
        assert torch.equal(out["dbeta"].double(), shown.double())
