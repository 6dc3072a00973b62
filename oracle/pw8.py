"""CPU oracle for the 8-bit pointwise convolution -- test infrastructure.

Only ``tests/`` may import this module; the product path never does.

The formulas are those that include/deft.h states for deft_pw8_*, in float64
torch on the inputs' device.  Every product of two coded values is exact there
and in the kernels, so what may differ is their sums: each result comes with
the sum of its terms' magnitudes, and the sum of the largest terms among each 8
consecutive ones (or a bound of it: the product of the factors' largest), by
which tests bound that.
"""
from __future__ import annotations

import torch

BLOCK = 128


def powers(most: torch.Tensor) -> torch.Tensor:
    """The least whole e >= -127 with most <= 448 * 2^e (float64)."""
    e = torch.floor(torch.log2(most.clamp(min=2.0 ** -300))) - 12
    while True:
        short = (most > 448 * torch.exp2(e)) | (e < -127)
        if not short.any():
            return e
        e = e + short


def nearest(q: torch.Tensor) -> torch.Tensor:
    """The nearest e4m3 values of |q| <= 448, ties to the even code."""
    a = q.abs()
    step = torch.full_like(a, 2.0 ** -9)
    for e in range(-6, 9):
        step = torch.where(a >= 2.0 ** e, torch.full_like(a, 2.0 ** (e - 3)), step)
    return torch.round(q / step) * step


def _pad(t: torch.Tensor, rows: int, depth: int) -> torch.Tensor:
    out = torch.zeros((-(-t.shape[0] // rows) * rows, -(-t.shape[1] // depth) * depth), dtype=torch.float64,
                      device=t.device)
    out[:t.shape[0], :t.shape[1]] = t
    return out


def coded(t: torch.Tensor, rows: int = 1, depth: int = BLOCK) -> torch.Tensor:
    """What t's codes stand for, in blocks of `rows` x `depth`; NaN where t is not finite."""
    p = _pad(t.double(), rows, depth)
    b = p.view(p.shape[0] // rows, rows, p.shape[1] // depth, depth)
    finite = torch.isfinite(b)
    scale = torch.exp2(powers(torch.where(finite, b, torch.zeros_like(b)).abs().amax((1, 3), keepdim=True)))
    v = torch.where(finite, nearest(torch.where(finite, b, torch.zeros_like(b)) / scale) * scale,
                    torch.full_like(b, float("nan")))
    return v.reshape(p.shape)[:t.shape[0], :t.shape[1]]


def product(a: torch.Tensor, b: torch.Tensor):
    """(a @ b, |a| @ |b|, sums over the groups of 8 terms of their largest magnitude, and of its square)."""
    def largest(t):
        t = _pad(torch.nan_to_num(t).abs(), 1, 8)
        return t.view(t.shape[0], -1, 8).amax(2)

    ga, gb = largest(a), largest(b.t().contiguous()).t()
    return a.mm(b), a.abs().mm(b.abs()), ga.mm(gb), ga.square().mm(gb.square())


def forward(x, w, b=None):
    """x [rows][c_in], w [c_out][c_in]: what product() gives, the bias added to the first two."""
    y, mag, group, square = product(coded(x), coded(w, BLOCK, BLOCK).t())
    if b is not None:
        y, mag = y + b.double(), mag + b.double().abs()
    return y, mag, group, square


def backward(x, w, dy):
    """dict of what product() gives (db: of the sum and the magnitudes)."""
    return dict(dx=product(coded(dy), coded(w, BLOCK, BLOCK)),
                dw=product(coded(dy.t()), coded(x.t()).t()),
                db=(dy.double().sum(0), dy.double().abs().sum(0)))
