"""What Muon's constructor refuses: tensors that share memory which a step writes, and rates that no step takes.
Without a GPU."""
import math

import pytest
import torch

from irregular_gather_cnn_amd import _lib as L
from irregular_gather_cnn_amd.optim import Muon


def tensors(dtype=torch.bfloat16):
    p = [torch.zeros(s, dtype=dtype) for s in ((4, 6), (3, 2, 4))]
    return p, [torch.zeros_like(t) for t in p]


def test_separate_tensors_are_taken():
    p, g = tensors()
    base = torch.zeros(96)
    Muon(p, g, masters=[base[:24], base[24:48]], states=[base[48:72], base[72:]])
    Muon(p, [g[0], g[0].view(3, 2, 4)])  # gradients are only read
    empty = [torch.zeros((0, 4)), torch.zeros((0, 4))]
    Muon([empty[0], empty[0]], empty, states=[empty[0], empty[0]])


@pytest.mark.parametrize("what", ["params", "states", "masters", "state and master", "state and param", "views"])
def test_shared_memory(what):
    p, g = tensors()
    one, base = torch.zeros(24), torch.zeros(40)
    more = dict(states=[torch.zeros(24), torch.zeros(24)], masters=[torch.zeros(24), torch.zeros(24)])
    if what == "params":
        p[1] = p[0]
    elif what == "states":
        more["states"] = [one, one]
    elif what == "masters":
        more["masters"] = [one, one]
    elif what == "state and master":
        more["states"][1] = more["masters"][0] = one
    elif what == "state and param":
        p, g = tensors(torch.float32)
        more = dict(states=[torch.zeros(24), p[0].view(-1)])
    else:  # neither starts where the other does
        more["states"] = [base[:24], base[16:]]
    with pytest.raises(ValueError, match="memory|twice"):
        Muon(p, g, **more)

@pytest.mark.parametrize("kw", [dict(steps=0), dict(steps=33), dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=math.nan),
                                dict(lr=-1.0), dict(lr=math.inf), dict(eps=0.0), dict(eps=math.nan)])
def test_rates(kw):
    with pytest.raises(L.DeftError):
        Muon(*tensors(), **kw)


@pytest.mark.parametrize("decay", [-0.1, math.nan, math.inf, [0.1, -0.1]])
def test_weight_decay(decay):
    with pytest.raises(ValueError, match="decay"):
        Muon(*tensors(), weight_decay=decay)


def test_masters_are_for_bf16():
    with pytest.raises(L.DeftError):
        Muon(*tensors(torch.float32), masters=[torch.zeros(24), torch.zeros(24)])
    with pytest.raises(ValueError):  # float32 copies of float32 params are the params
        Muon(*tensors(torch.float32), masters=True)
