"""Oracle for the group norm with activation on large inputs -- test infrastructure.

Only ``tests/`` may import this module; the product path never does.

The formulas of ``oracle/norm.py`` in torch float64, on the inputs' device, and
for the forward bounds that follow its own sums: ``accesses`` of ``vec`` elements
a thread in fp32, then fp64, then one rounding of each slice's and each group's
mean.  (The backward sums in fp32 throughout; its bounds are those of
``oracle/norm.py``.)
"""
from __future__ import annotations

import math

import torch

from .norm import CURVE, H, K, TAIL


def act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0 * z)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z


def _density(z):
    return torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def slope(name, z):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return torch.special.ndtr(z) + z * _density(z)
    return torch.ones_like(z)


def own_act_error(name, z, y, dtype):
    a = z.abs()
    if name == "silu":
        return y.abs() * (2 * a + 8) * H
    if name == "gelu":
        return a * torch.special.ndtr(-a) * (TAIL[dtype] + (2 * z * z + 8) * H) + 4 * H * y.abs()
    return 0 * a


def own_slope_error(name, z, dtype):
    a = z.abs()
    if name == "silu":
        p = torch.sigmoid(z)
        return (p + p * a * (1 - p) + a * p * p) * (2 * a + 10) * H
    if name == "gelu":
        return (torch.special.ndtr(-a) * (TAIL[dtype] + (2 * z * z + 8) * H)
                + a * _density(z) * (2 * z * z + 8) * H + 4 * H)
    return 0 * a


def forward(x, gamma, beta, g, eps, name, dtype, accesses, vec):
    """dict of (value, bound) for y, mean, rstd of float64 x [n][c][s]; y's bound without its last rounding."""
    n, c, s = x.shape
    xg = x.reshape(n, g, -1)
    size, most = xg.abs().mean(2), xg.abs().amax(2)
    mean = xg.mean(2)
    var = (xg - mean[:, :, None]).square().mean(2)
    std, squares = var.sqrt(), xg.square().mean(2)
    rstd = (var + eps).rsqrt()
    # one thread's sum: an addition an access and the joining of its columns; bf16 two in an access,
    # of an instruction that may cut off (2 H) where others round
    chain = (accesses if dtype == "f32" else 4 * accesses) + 8
    e_mean = (chain + 2) * H * size + H * mean.abs()
    if dtype == "f32":
        # squares about each thread's own mean, which then counts by its distance from the group's: that
        # distance sums to at most a standard deviation an element
        e_var = (accesses * vec + 12) * H * var + 2 * std * (chain + 1) * H * most
    else:
        # plain squares
        e_var = chain * H * squares + 2 * mean.abs() * e_mean + 2 * std * H * most + 4 * H * var
    e_var = e_var + e_mean * e_mean + 1e-14 * squares
    r_rstd = 0.5 * e_var / (var + eps) + 6 * H

    def wide(v):
        return v.repeat_interleave(c // g, dim=1)[:, :, None]

    ga, be = gamma[None, :, None], beta[None, :, None]
    d, rs = x - wide(mean), wide(rstd)
    z = d * rs * ga + be
    ez = ga.abs() * rs * (wide(e_mean) + 2 * H * d.abs()) + (ga * rs * d).abs() * (wide(r_rstd) + 3 * H) + H * z.abs()
    y = act(name, z)
    return dict(y=(y, 1.13 * ez + own_act_error(name, z, y, dtype)), mean=(mean, e_mean), rstd=(rstd, r_rstd * rstd))


def backward(x, gamma, beta, mean, rstd, dy, g, name, dtype):
    """dict of (value, bound) for dx, dgamma, dbeta from given mean and rstd [n][g]."""
    n, c, s = x.shape

    def wide(v):
        return v.repeat_interleave(c // g, dim=1)[:, :, None]

    def group(v):
        return v.reshape(n, g, -1).sum(2)

    mu, rs = wide(mean), wide(rstd)
    ga, be = gamma[None, :, None], beta[None, :, None]
    m = c // g * s
    h = (x - mu) * rs
    z = h * ga + be
    dz = dy * slope(name, z)
    ez = 5 * H * (h * ga).abs() + 2 * H * z.abs()
    e_dz = dy.abs() * (CURVE[name] * ez + own_slope_error(name, z, dtype)) + 2 * H * dz.abs()
    if name == "relu":  # either side of the corner
        e_dz = e_dz + dy.abs() * (z.abs() <= ez)
    a, b = dz.sum(2), (dz * h).sum(2)
    ea = e_dz.sum(2) + K * H * dz.abs().sum(2)
    eb = (e_dz * h.abs()).sum(2) + (K + 4) * H * (dz * h).abs().sum(2)
    gc = gamma[None, :]
    s1, s2 = group(gc * a), group(gc * b)
    es1 = group(gc.abs() * ea) + K * H * group((gc * a).abs())
    es2 = group(gc.abs() * eb) + K * H * group((gc * b).abs())
    dx = rs * (ga * dz - wide(s1) / m - h * wide(s2) / m)
    e_dx = (rs * ga.abs() * (e_dz + 4 * H * dz.abs()) + rs / m * (wide(es1) + 6 * H * wide(s1).abs())
            + rs / m * h.abs() * (wide(es2) + 10 * H * wide(s2).abs()) + 2 * H * dx.abs())
    return dict(dx=(dx, e_dx), dgamma=(b.sum(0), eb.sum(0) + K * H * b.abs().sum(0)),
                dbeta=(a.sum(0), ea.sum(0) + K * H * a.abs().sum(0)))
