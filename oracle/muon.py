"""CPU oracle for the Muon step -- test infrastructure.

Only ``tests/`` may import this module; the product path never does.

The formulas are those that include/deft.h states for deft_muon_step: the
update's direction in float64 torch on the inputs' device, momentum and weights
in fp32 with one rounding per operation.
"""
from __future__ import annotations

import torch

A, B, C = 3.4445, -4.7750, 2.0315
# the steepest slope of sigma -> A sigma + B sigma^3 + C sigma^5 over |sigma| <= 1.21: at the ends
STEEPEST = A + 3 * B * 1.21 ** 2 + 5 * C * 1.21 ** 4


def orthogonal(u: torch.Tensor, steps: int, eps: float = 1e-7):
    """(X, sizes): the direction after `steps`, and what an error of relative size 1 at each step comes to in
    it, in Frobenius norms: sum over k of STEEPEST^(steps - k) |X_k|."""
    x = u.double()
    x = x / torch.linalg.vector_norm(x).clamp(min=eps)
    sizes = 0.0
    for k in range(steps):
        sizes = STEEPEST * sizes + float(torch.linalg.vector_norm(x)) * STEEPEST
        g = x.mm(x.t()) if x.shape[0] <= x.shape[1] else x.t().mm(x)
        q = B * g + C * g.mm(g)
        q.diagonal().add_(A)
        x = q.mm(x) if x.shape[0] <= x.shape[1] else x.mm(q)
    return x, sizes + float(torch.linalg.vector_norm(x))


def momentum(m, g, mu, nesterov, coef=None):
    """(m, u) in fp32, one rounding per operation."""
    one = torch.tensor(1.0, dtype=torch.float32, device=m.device)
    a, b = one * mu, one * (1.0 - mu)
    g = g.float() if coef is None else g.float() * coef
    m = m * a + g * b
    return m, (m * a + g * b if nesterov else m)


def update(p, x, lr, weight_decay, scale):
    """p in fp32 after the step along x (fp32)."""
    one = torch.tensor(1.0, dtype=torch.float32, device=p.device)
    return p.float() * (one * (1.0 - lr * weight_decay)) - x * (one * (lr * scale))
