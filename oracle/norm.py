"""CPU oracle for the group norm with activation -- test infrastructure.

Only ``tests/`` may import this module; the product path never does.

The formulas of include/deft.h (deft_norm_forward, deft_norm_backward) in
float64 on channels-first arrays [n][c][s], with bounds on what fp32 sums and
roundings may add to them.  Forward, a thread sums up to 32 accesses in fp32
(``CHAIN``: an addition each, two in bf16, which may cut off where others round,
and 8 more that join its columns); beyond it all sums are fp64, and each slice's
mean is rounded once.  Backward, ``K`` counts the longest chain of fp32 additions
that a value passes through: 64 rows or 128 elements of a thread, at most 22 that
join threads, 16 waves, then slices or images in shares of 64 with 20 to join them.
"""
from __future__ import annotations

import math

import numpy as np
from scipy.special import ndtr

H = 2.0 ** -24
K = 256
CHAIN = {"f32": 40, "bf16": 136}


def act(name, z):
    if name == "relu":
        return np.where(np.isnan(z), z, np.maximum(z, 0))
    if name == "silu":
        return z / (1 + np.exp(-z))
    if name == "gelu":
        return z * ndtr(z)
    return z


def slope(name, z):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        p = 1 / (1 + np.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return ndtr(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return np.ones_like(z)


# relative error of the kernels' normal tail: its fit and, fp32, its roundings
TAIL = {"f32": 6e-7, "bf16": 6e-6}


def _groups(x, g):
    n, c, s = x.shape
    return x.reshape(n, g, -1)


def _per_channel(v, n, c):
    """[n][g] -> [n][c][1]"""
    return np.repeat(v, c // v.shape[1], axis=1)[:, :, None]


def forward(x, gamma, beta, g, eps, name, dtype):
    """dict of (value, bound) for y, mean, rstd; y's bound without its last rounding."""
    n, c, s = x.shape
    xg = _groups(x, g)
    m = xg.shape[2]
    mean = xg.mean(2)
    d = xg - mean[:, :, None]
    m2 = (d * d).sum(2)
    var = m2 / m
    rstd = 1 / np.sqrt(var + eps)
    size, std = np.abs(xg).mean(2), np.sqrt(var)
    e_mean = (CHAIN[dtype] + 2) * H * size + H * np.abs(mean)
    # d is rounded and off by the mean's error: the sum of d is zero, so that counts squared
    e_var = (K + 8) * H * var + (K * H * size + H * np.abs(mean) + 2 * H * size) ** 2 * 2
    if dtype == "f32":
        # or: squares about each thread's own mean, which then counts by its distance from the group's
        e_var = np.minimum(e_var, 140 * H * var + 2 * std * (CHAIN[dtype] + 1) * H * np.abs(xg).max(2) + e_mean ** 2)
    r_rstd = 0.5 * e_var / (var + eps) + 4 * H
    mu, rs = _per_channel(mean, n, c), _per_channel(rstd, n, c)
    em, rr = _per_channel(e_mean, n, c), _per_channel(r_rstd, n, c)
    ga, be = gamma[None, :, None], beta[None, :, None]
    dd = x - mu
    z = dd * rs * ga + be
    ez = np.abs(ga) * rs * (em + 2 * H * np.abs(dd)) + np.abs(ga * rs * dd) * (rr + 4 * H) + 2 * H * np.abs(z)
    y = act(name, z)
    ey = 1.13 * ez + own_act_error(name, z, y, dtype)
    return dict(y=(y, ey), mean=(mean, e_mean), rstd=(rstd, r_rstd * rstd))


def own_act_error(name, z, y, dtype):
    a = np.abs(z)
    if name == "silu":
        return np.abs(y) * (2 * a + 8) * H
    if name == "gelu":
        return a * ndtr(-a) * (TAIL[dtype] + (2 * z * z + 8) * H) + 4 * H * np.abs(y)
    return 0 * a


def own_slope_error(name, z, dtype):
    a = np.abs(z)
    if name == "silu":
        p = 1 / (1 + np.exp(-z))
        return (p + p * a * (1 - p) + a * p * p) * (2 * a + 10) * H
    if name == "gelu":
        phi = np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return ndtr(-a) * (TAIL[dtype] + (2 * z * z + 8) * H) + a * phi * (2 * z * z + 8) * H + 4 * H
    return 0 * a


# largest |second derivative|
CURVE = {"none": 0.0, "relu": 0.0, "silu": 0.5, "gelu": 0.8}


def backward(x, gamma, beta, mean, rstd, dy, g, name, dtype):
    """dict of (value, bound) for dx, dgamma, dbeta from given mean and rstd [n][g]."""
    n, c, s = x.shape
    mu, rs = _per_channel(mean, n, c), _per_channel(rstd, n, c)
    ga, be = gamma[None, :, None], beta[None, :, None]
    m = c // g * s
    d = x - mu
    h = d * rs
    z = h * ga + be
    dz = dy * slope(name, z)
    ez = 5 * H * np.abs(h * ga) + 2 * H * np.abs(z)
    e_dz = np.abs(dy) * (CURVE[name] * ez + own_slope_error(name, z, dtype)) + 2 * H * np.abs(dz)
    if name == "relu":  # either side of the corner
        e_dz = e_dz + np.abs(dy) * (np.abs(z) <= ez)
    a = dz.sum(2)
    ea = e_dz.sum(2) + K * H * np.abs(dz).sum(2)
    b = (dz * h).sum(2)
    eb = (e_dz * np.abs(h)).sum(2) + (K + 4) * H * np.abs(dz * h).sum(2)
    gc = gamma[None, :]
    dbeta, e_dbeta = a.sum(0), ea.sum(0) + K * H * np.abs(a).sum(0)
    dgamma, e_dgamma = b.sum(0), eb.sum(0) + K * H * np.abs(b).sum(0)

    def group(v):
        return v.reshape(n, g, -1).sum(2)

    s1, s2 = group(gc * a), group(gc * b)
    es1 = group(np.abs(gc) * ea) + K * H * group(np.abs(gc * a))
    es2 = group(np.abs(gc) * eb) + K * H * group(np.abs(gc * b))
    p = lambda v: _per_channel(v, n, c)  # noqa: E731
    dx = rs * (ga * dz - p(s1) / m - h * p(s2) / m)
    e_dx = (rs * np.abs(ga) * (e_dz + 4 * H * np.abs(dz)) + rs / m * (p(es1) + 6 * H * np.abs(p(s1)))
            + rs / m * np.abs(h) * (p(es2) + 10 * H * np.abs(p(s2))) + 2 * H * np.abs(dx))
    return dict(dx=(dx, e_dx), dgamma=(dgamma, e_dgamma), dbeta=(dbeta, e_dbeta))
