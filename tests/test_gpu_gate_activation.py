"""The gate's activation over the whole range of FP32, through the gated calls.

The operands make the gate sum a chosen number exactly (codes with sum 1, a scale
per token) and the up sum that number times a constant, so that a call's only
inexact steps are those of its epilogue.  Tolerances (u = 2^-24, y the logistic
function's argument; from the calls' own statements):
  int8, FP32 out   8 u |act| + 2^-128 |x| + 2^-149, times |up|; up and the last
                   product round three times, 3 u |h|
  BF16 out, E4M3   (16 + 8 |y|) u |act| in place of 8 u |act|
  h                half an ulp of BF16, and 2^-149, of the stored value
"""

import numpy as np
import pytest
import torch

from gpu_util import DEV, fq
from oracle import gemm as ogemm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LD = np.longdouble


def _gates():
    """FP32 values: small and large ones of both signs, 1 to 100 densely, the ends
    of the exponential's range."""
    rng = np.random.default_rng(1)
    tiny = 2.0 ** np.arange(-126, -8, 2.37) * 1.3
    x = np.concatenate([tiny, rng.uniform(0.004, 1, 60), rng.uniform(1, 12, 200),
                        rng.uniform(12, 100, 150), np.linspace(86, 90, 41),
                        2.0 ** np.arange(7, 105, 4.1)])
    return np.concatenate([x, -x]).astype(np.float32)


def _exact(act, x):
    x = x.astype(LD)
    c = 2 * np.sqrt(LD(2) / LD(np.pi))
    y = x if act == "silu" else c * (x + LD("0.044715") * x ** 3)
    with np.errstate(over="ignore"):
        return x / (1 + np.exp(-y)), y


def _hold(h, x, up, act, exact_form):
    """h [M][F] against act(x[m]) * up[m][f]; up is that of the operands in longdouble.
    Pairs whose up or h leaves the normal range are left out."""
    a, y = _exact(act, x)
    a, y, xl = a[:, None], y[:, None], np.abs(x.astype(LD))[:, None]
    ref = a * up
    live = (np.abs(up) > 2.0 ** -120) & (np.abs(up) < 2.0 ** 120) & (np.abs(ref) < 2.0 ** 127)
    assert live.any(axis=1).all()               # every gate is held somewhere
    rel = 8 if exact_form else 16 + 8 * np.abs(y)
    tol = (rel * U * np.abs(a) + LD(2) ** -128 * xl + LD(2) ** -149) * np.abs(up) \
        + 3 * U * np.abs(ref) + LD(2) ** -149
    if h.dtype == torch.bfloat16:
        tol = tol + ogemm.bf16_half_ulp(ref.astype(np.float64)) * (1 + 2.0 ** -6) + LD(2) ** -133
    err = np.abs(h.double().cpu().numpy().astype(LD) - ref)
    assert (err <= tol)[live].all(), (x[np.argwhere((err > tol) & live)[:, 0]][:8])


# 16 rows: the kernel for few rows; all of them, with many columns: a tile
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("F,few", [(5, True), (2000, False)])
def test_int8(act, out, F, few):
    x = _gates()
    K = 16
    a = np.full((len(x), K), 127, dtype=np.int8)
    a[:, 0] = 1
    w = np.zeros((2 * F, K), dtype=np.int8)
    w[:F, 0] = 1                                # gate sums: 1
    w[F:, 1:] = 127                             # up sums: 15 * 127 * 127
    ws = np.ones(2 * F, dtype=np.float32)
    ws[F:] = np.array([2.0 ** -16, 2.0 ** 100, 2.0 ** -60, 2.0 ** -110, 2.0 ** 50])[np.arange(F) % 5]
    dev = [torch.from_numpy(v).to(DEV) for v in (a, x, w, ws)]
    up = (15 * 127 * 127) * x.astype(LD)[:, None] * ws[None, F:].astype(LD)
    step = 16 if few else len(x)
    for r in range(0, len(x), step):
        h = fq().gemm_i8_gated(dev[0][r:r + step], dev[1][r:r + step], dev[2], dev[3], act=act,
                               out_dtype=out)
        _hold(h, x[r:r + step], up[r:r + step], act, out == torch.float32)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("few", [True, False])
def test_e4m3(act, out, few):
    x = _gates()
    K, F, one = 128, 5 * 128, 0x38
    a = np.full((len(x), K), one, dtype=np.uint8)
    w = np.zeros((2 * F, K), dtype=np.uint8)
    w[:F, 0] = one                              # gate sums: 1
    w[F:] = one                                 # up sums: 128
    ws = np.ones((2 * F // 128, 1), dtype=np.float32)
    ws[F // 128:, 0] = [2.0 ** -16, 2.0 ** 100, 2.0 ** -60, 2.0 ** -110, 2.0 ** 50]
    dev = [torch.from_numpy(v).to(DEV) for v in (a, x[None, :], w, ws)]
    up = 128 * x.astype(LD)[:, None] * np.repeat(ws[F // 128:, 0], 128)[None, :].astype(LD)
    step = 16 if few else len(x)
    for r in range(0, len(x), step):
        h = fq().gemm_gated(dev[0][r:r + step].contiguous(), dev[1][:, r:r + step].contiguous(),
                            dev[2], dev[3], act=act, out_dtype=out)
        _hold(h, x[r:r + step], up[r:r + step], act, False)
