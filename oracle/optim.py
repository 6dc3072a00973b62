"""CPU oracle for the gradient norm and the AdamW step -- test infrastructure.

Only ``tests/`` may import this module; the product path never does.

The formulas are those that include/deft.h states for deft_adamw_step and
deft_grad_norm, element by element in numpy.  ``dt`` chooses the arithmetic:
float64 gives the value of the formulas, float32 the bits of a step that rounds
every operation once in the stated order.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 256


def e4m3_values() -> np.ndarray:
    """The 127 finite non-negative e4m3 values in the order of their codes (0 .. 0x7e)."""
    code = np.arange(0x7F)
    exp, frac = code >> 3, code & 7
    return np.where(exp == 0, frac * 2.0 ** -9, (8 + frac) * 2.0 ** (exp - 10.0))


def decode(codes: np.ndarray) -> np.ndarray:
    """uint8 e4m3 codes -> float64 (0x7f and 0xff are NaN)."""
    table = np.append(e4m3_values(), np.nan)
    c = np.asarray(codes, np.uint8)
    return np.where(c & 0x80, -1.0, 1.0) * table[c & 0x7F]


def encode_nearest(t: np.ndarray) -> np.ndarray:
    """Codes of the nearest values, ties to the even code; |t| <= 448."""
    v = e4m3_values()
    a = np.abs(np.asarray(t, np.float64))
    hi = np.clip(np.searchsorted(v, a), 1, len(v) - 1)
    lo = hi - 1
    up = (a - v[lo] > v[hi] - a) | ((a - v[lo] == v[hi] - a) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(t), 0x80, 0)).astype(np.uint8)


def encode_random(t: np.ndarray, u16: np.ndarray) -> np.ndarray:
    """Codes of t in [0, 448] cut off after (u16 + 1/2) / 65536 of the code's step is added;
    what is not zero keeps the least code.  t is fp32: below 2^-6 the sum is one fp32 addition,
    as stated for the kernel; above, the random number is added to its 20 lower fraction bits."""
    v = e4m3_values()
    t = np.asarray(t, np.float32)
    bits = t.view(np.uint32) + (u16.astype(np.uint32) * np.uint32(16) + np.uint32(8))
    normal = (bits & np.uint32(0xFFF00000)).view(np.float32)
    u = (u16.astype(np.float32) + np.float32(0.5)) * np.float32(2.0 ** -16)
    small = np.floor(t * np.float32(512) + u) / np.float32(512)
    small = np.where(t > 0, np.maximum(small, np.float32(2.0 ** -9)), small)
    return np.searchsorted(v, np.where(t < 2.0 ** -6, small, normal)).astype(np.uint8)


def mix(x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, np.uint64) & 0xFFFFFFFF
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0xBB67AE85)) & np.uint64(0xFFFFFFFF)
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0x6A09E667)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def rounding_bits(n: int, tensor: int, seed: int) -> np.ndarray:
    """16 random bits for each of n elements of tensor number `tensor`."""
    key = mix(np.uint64((seed + tensor * 0x3C6EF373) & 0xFFFFFFFF))
    i = np.arange(n, dtype=np.uint64)
    h = mix((i >> np.uint64(1)) * np.uint64(0x6A09E667) + key)
    return ((h >> (np.uint64(16) * (i & np.uint64(1)))) & np.uint64(0xFFFF)).astype(np.uint32)


def quantise(a: np.ndarray, bits_of=None):
    """fp32 values of one tensor -> (codes, scales); bits_of: random bits (sqrt(v)) or None (m)."""
    a = np.asarray(a, np.float32)
    n = a.size
    codes, scales = np.zeros(n, np.uint8), np.zeros(-(-n // BLOCK), np.float32)
    for b in range(scales.size):
        sl = slice(b * BLOCK, min(n, (b + 1) * BLOCK))
        most = np.abs(a[sl]).max() if not np.isnan(a[sl]).any() else np.float32(np.nan)
        if not np.isfinite(most):
            scales[b] = np.nan
            continue
        s = most / np.float32(448)
        if s < np.float32(2.0 ** -126):
            continue
        scales[b] = s
        t = a[sl] * (np.float32(1) / s)
        if bits_of is None:
            codes[sl] = encode_nearest(np.clip(t, -448, 448))
        else:
            codes[sl] = encode_random(np.minimum(t, np.float32(448)), bits_of[sl])
    return codes, scales


def dequantise(codes, scales):
    """fp32 code * scale (one rounding)."""
    n = len(codes)
    with np.errstate(invalid="ignore"):
        return decode(codes).astype(np.float32) * np.repeat(np.asarray(scales, np.float32), BLOCK)[:n]


def adamw(p, g, m, v, *, step, lr, beta1, beta2, eps, weight_decay, coef=None, dt=np.float64):
    """(p, m, v, sqrt(v)) after the step, every operation in `dt`."""
    f = dt
    p, g, m, v = (np.asarray(a).astype(f) for a in (p, g, m, v))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if coef is not None:
            g = g * f(coef)
        m = m * f(beta1) + g * f(1.0 - beta1)
        v = v * f(beta2) + (g * g) * f(1.0 - beta2)
        root = np.sqrt(v)
        low, rate = f(1.0 / math.sqrt(1.0 - beta2 ** step)), f(lr / (1.0 - beta1 ** step))
        p = p * f(1.0 - lr * weight_decay) - (m / (root * low + f(eps))) * rate
    return p, m, v, root


def grad_norm(grads, max_norm, inv_scale):
    """(norm, factor, finite) in float64."""
    total = math.fsum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads)
    norm = math.sqrt(total) * inv_scale if math.isfinite(total) else total
    if not math.isfinite(norm):
        return norm, 0.0, 0.0
    f = 1.0 if math.isinf(max_norm) else min(1.0, max_norm / (norm + 1e-6))
    return norm, inv_scale * f, 1.0
