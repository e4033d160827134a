"""The operators of a training step around the products: layer norm, tokens
grouped by expert, AdamW.

TEST INFRASTRUCTURE ONLY (see the package docstring).

    layer_norm, layer_norm_backward   float64
    expert_blocks                     the groups of 128 tokens of each expert
    expert_rows                       x's rows in those groups, zeros between
    adamw_moments                     m and v in the FP32 operations the call names
    adamw_parameters                  p in float64 from given moments
    decode_moments, encode_moments    E4M3 moments, bit for bit: the dithered codes
"""

import numpy as np

from . import e4m3

F32 = np.float32


def layer_norm(x, weight, bias, eps):
    """float64 (y, mean, rstd) of rows x[M][N]."""
    x = x.astype(np.float64)
    mean = x.mean(axis=1)
    var = ((x - mean[:, None]) ** 2).mean(axis=1)
    rstd = 1.0 / np.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None] * weight.astype(np.float64)
    return y + (0.0 if bias is None else bias.astype(np.float64)), mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd):
    """float64 (dx, dweight, dbias), with mean and rstd as given."""
    dy, x, w = (t.astype(np.float64) for t in (dy, x, weight))
    r = rstd.astype(np.float64)[:, None]
    z = (x - mean.astype(np.float64)[:, None]) * r
    gz = dy * w
    dx = r * (gz - gz.mean(axis=1, keepdims=True) - z * (gz * z).mean(axis=1, keepdims=True))
    return dx, (dy * z).sum(axis=0), dy.sum(axis=0)


def expert_blocks(off):
    """[(expert, first row, rows, first column)] of every group of 128 tokens."""
    out = []
    for e in range(len(off) - 1):
        for r in range(off[e], off[e + 1], 128):
            out.append((e, r, min(128, off[e + 1] - r), 128 * len(out)))
    return out


def expert_rows(x, off, columns):
    """x[M][K] -> [columns][K]: each group's rows from its first column on."""
    out = np.zeros((columns, x.shape[1]), dtype=x.dtype)
    for _, r, n, c in expert_blocks(off):
        out[c:c + n] = x[r:r + n]
    return out


def adamw_moments(m, v, g, beta1, beta2):
    """(m', v') in float32, each operation rounded once."""
    m, v, g = (np.asarray(t, dtype=F32) for t in (m, v, g))
    m2 = m * F32(beta1) + g * F32(1.0 - beta1)
    v2 = v * F32(beta2) + (g * g) * F32(1.0 - beta2)
    return m2, v2


def adamw_parameters(p, m, v, step, lr, beta1, beta2, eps, weight_decay):
    """float64 (p', the update taken off it) from the new moments."""
    p, m, v = (t.astype(np.float64) for t in (p, m, v))
    c1 = -np.expm1(step * np.log(beta1)) if beta1 else 1.0
    c2 = -np.expm1(step * np.log(beta2)) if beta2 else 1.0
    update = lr / c1 * m / (np.sqrt(v) / np.sqrt(c2) + eps)
    return p * (1.0 - lr * weight_decay) - update, update


def _grouped(x):
    n = x.size
    return np.concatenate([x, np.zeros(-n % 128, dtype=x.dtype)]).reshape(-1, 128)


def decode_moments(codes, scales):
    """float32 [n] = fl(code * scale)."""
    n = codes.size
    x = e4m3.decode(codes).astype(F32) * np.repeat(scales.astype(F32), 128)[:n]
    return x.astype(F32)


def dither(n, step, second=False, first=0):
    """The 20 bits of elements first .. first + n - 1."""
    i = np.arange(first, first + n, dtype=np.uint64)
    u = i * np.uint64(0x85EBCA6B) + np.uint64(step * 0x9E3779B1 % 2 ** 32)   # (mod 2^64)
    u = ((u & np.uint64(0xFFFFFFFF)) >> np.uint64(12)).astype(np.int64)
    return 0xFFFFF - u if second else u


def encode_moments(x, step, second=False, first=0):
    """(codes, scales) of float32 x[n] (second: a root, >= 0), bit for bit; x[0] is
    element `first` of its tensor.  What is not finite gets the code of NaN and has no
    part in its group's scale."""
    x = np.asarray(x, dtype=F32)
    n = x.size
    finite = np.isfinite(x)
    x = np.where(finite, x, F32(0))
    amax = np.abs(_grouped(x)).max(axis=1)
    with np.errstate(divide="ignore", over="ignore"):
        mul = F32(448) * (F32(1) / amax)
    flush = ~np.isfinite(mul)
    mul = np.where(flush, F32(0), mul)
    scales = np.where(flush, F32(0), amax * (F32(1) / F32(448)))
    y = x * np.repeat(mul, 128)[:n]
    a = np.abs(y)
    sub = a < F32(2.0 ** -6)
    b = np.where(sub, a + F32(2.0 ** -6), a).astype(F32)
    bits = (b.view(np.int32).astype(np.int64) + dither(n, step, second, first)) & ~np.int64(0xFFFFF)
    r = bits.astype(np.int32).view(F32)
    r = np.minimum(np.where(sub, r - F32(2.0 ** -6), r), F32(448))
    if second:
        r = np.where((r == 0) & (a > 0), F32(2.0 ** -9), r)
    codes = e4m3.encode(r.astype(np.float64))   # (exact: r is an E4M3 value)
    codes = np.where(np.signbit(y), codes | 0x80, codes)
    return np.where(finite, codes, 0x7F).astype(np.uint8), scales.astype(F32)
