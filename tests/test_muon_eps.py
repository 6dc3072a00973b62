"""Muon's directions far below eps.

X is held in multiples of 2^-38 (pairs of fp16 times 2^14, whose least part is 2^-24), so besides what the other tests
bound, each of its elements may be off by half of that, which each step multiplies by at most A; X is rounded so at
the start and once for each product with it, at most three times where the first counts most: 3 A^5 2^-39 of the root
of the number of elements."""
import math

import pytest
import torch

from oracle import muon as O
from test_muon import direction, rand
from test_muon_tiles import bound


@pytest.mark.gpu
@pytest.mark.parametrize("below", [0, 3, 5, 7, 9, 11, 14])
@pytest.mark.parametrize("shape", [(40, 90), (300, 1000), (1100, 4003)])
def test_directions_far_below_eps(shape, below):
    eps = 1e-7
    u = rand(shape, 3)
    u *= eps * 10.0 ** -below / float(u.double().norm())
    print("muon eps", shape, below, flush=True)
    x = direction([u], eps=eps)[0]
    want, _ = O.orthogonal(u, 5, eps)
    # steps in fp32 of u / |u| are off by as much of X as those of u / eps, or more
    unit, _ = O.orthogonal(u, 5, 1e-300)
    plain = bound(u, unit)[0] / float(unit.norm()) * float(want.norm())
    allowed = 4 * plain + 2.0 ** -22 * float(want.norm()) + 3 * O.A ** 5 * 2.0 ** -39 * math.sqrt(u.numel())
    off = float((x.double() - want).norm())
    print("  off %.2e of %.2e, allowed %.2e" % (off, float(want.norm()), allowed), flush=True)
    assert off <= allowed
