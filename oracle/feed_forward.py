"""The 8-bit feed-forward layer, evaluated in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

    quantize_token_i8   one scale per row, int8 codes (FP32 multiplier, as stated
                        by the call's rule, so the codes are determined)
    gemm_i8             integer product, exact, scaled in float64
    act, act_grad       SiLU and the tanh form of GELU, and their derivatives
    gated               act(gate) * up of [gate | up]
    gated_backward      dY = [dh up act'(gate) | dh act(gate)]

act is written with the logistic function (1 + tanh z = 2 sigma(2z)), which
keeps the relative accuracy of a small result.
"""

import numpy as np


def quantize_token_i8(x):
    """x: float32[M][K] (BF16 values) -> (int8[M][Kp], float32[M])."""
    x = np.asarray(x, dtype=np.float32)
    M, K = x.shape
    amax = np.abs(x).max(axis=1)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.float32(127) * (np.float32(1) / amax)
    flush = ~np.isfinite(inv)
    inv = np.where(flush, np.float32(0), inv)
    q = np.zeros((M, -(-K // 16) * 16), dtype=np.int8)
    q[:, :K] = np.clip(np.rint(x * inv[:, None]), -127, 127).astype(np.int8)
    return q, np.where(flush, np.float32(0), amax / np.float32(127))


def gemm_i8(qa, sa, qw, sw):
    """float64[M][N]: the integer product (exact: below 2^31), scaled."""
    p = qa.astype(np.float64) @ qw.astype(np.float64).T
    return p * sa.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]


def act_arg(act, x):
    """y with act(x) = x sigma(y)."""
    if act == "silu":
        return x
    return 2.0 * np.sqrt(2.0 / np.pi) * (x + 0.044715 * x ** 3)


def _sigma(y):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-y))


def act(name, x):
    x = np.asarray(x, dtype=np.float64)
    return x * _sigma(act_arg(name, x))


def act_grad(name, x):
    x = np.asarray(x, dtype=np.float64)
    y = act_arg(name, x)
    dy = 1.0 if name == "silu" else 2.0 * np.sqrt(2.0 / np.pi) * (1.0 + 3 * 0.044715 * x ** 2)
    return _sigma(y) + x * dy * _sigma(y) * _sigma(-y)


def gated(name, Y):
    F = Y.shape[1] // 2
    return act(name, Y[:, :F]) * Y[:, F:]


def gated_backward(name, dh, Y):
    """float64 [M][2F] = [dgate | dup]."""
    F = dh.shape[1]
    dh, g, u = dh.astype(np.float64), Y[:, :F].astype(np.float64), Y[:, F:].astype(np.float64)
    return np.concatenate([dh * u * act_grad(name, g), dh * act(name, g)], axis=1)
