"""Sizes that do not fit the descriptors' 32 bits are refused, not cut to their low bits.  Without a GPU."""
import pytest
import torch

from irregular_gather_cnn_amd import _lib as L
from irregular_gather_cnn_amd.norm import GroupNormAct
from irregular_gather_cnn_amd.optim import Muon
from irregular_gather_cnn_amd.pointwise import Pointwise8

BEYOND = [1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 31) - 1, (1 << 64) + 5]


@pytest.mark.parametrize("size", BEYOND)
@pytest.mark.parametrize("which", ["n", "s", "c_in", "c_out"])
def test_pointwise(which, size):
    with pytest.raises(ValueError, match=which):
        Pointwise8(**{**dict(n=1, s=8, c_in=8, c_out=8), which: size}, device="cpu")


@pytest.mark.parametrize("size", BEYOND)
@pytest.mark.parametrize("which", ["n", "c", "s", "groups"])
def test_group_norm(which, size):
    with pytest.raises(ValueError, match=which):
        GroupNormAct(**{**dict(n=1, c=8, s=8, groups=8), which: size}, device="cpu")


@pytest.mark.parametrize("size", BEYOND)
def test_muon_steps(size):
    with pytest.raises(ValueError, match="steps"):
        Muon([torch.zeros(4, 6)], [torch.zeros(4, 6)], steps=size)


@pytest.mark.parametrize("size", BEYOND)
def test_deformable_layer(size):
    with pytest.raises(ValueError, match="c_in"):
        L.make_desc(1, size, 8, 8, 8)


def test_sizes_that_fit_are_left_to_the_library():
    assert L.deft_pw8_desc(1, (1 << 31) - 1, 8, 8, 1, 1, 0).s == (1 << 31) - 1
    assert L.deft_pw8_desc(-(1 << 31), 8, 8, 8, 1, 1, 0).n == -(1 << 31)
    with pytest.raises(L.DeftError):  # more positions than the kernels count
        Pointwise8(1, 8, (1 << 31) - 1, 8, device="cpu")
