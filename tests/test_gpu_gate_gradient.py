"""The gated backward pass's dgate and dup for every finite BF16 gate, to the bound
that its declaration states.

A group's scale is the FP32 quotient of its largest |dY| by 448.  With one token's
dh = up = 1 alone in a group the scale therefore shows |act'(gate)| and |act(gate)|
to an FP32 unit, where the codes show three bits of them.
"""

import numpy as np
import pytest
import torch

from gpu_util import DEV, fq, host, to_dev_bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LD = np.longdouble


def _gates():
    """Every finite BF16 value: (bits, values)."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    return bits, (bits.astype(np.uint32) << 16).view(np.float32)


def _exact(act, x):
    """act(x), act'(x) and the bounds of their errors, in longdouble."""
    x = x.astype(LD)
    c = 2 * np.sqrt(LD(2) / LD(np.pi))
    y = x if act == "silu" else c * (x + LD("0.044715") * x ** 3)
    dy = 1 if act == "silu" else c * (1 + 3 * LD("0.044715") * x ** 2)
    with np.errstate(over="ignore"):
        s, t = 1 / (1 + np.exp(-y)), 1 / (1 + np.exp(y))
    a, da = x * s, s + x * dy * s * t
    rel = (16 + 8 * np.minimum(np.abs(y), 100)) * U
    return a, da, rel * np.abs(a) + 2.0 ** -119, rel * (np.abs(da) + np.abs(x * dy * s * t)) + 2.0 ** -119


def _hold(scales, ref, bound):
    got = host(scales).astype(LD) * 448
    ref = np.abs(ref)
    # the quotient's rounding, to a unit of the smallest FP32 numbers at least
    err, tol = np.abs(got - ref), bound + U * ref + 448 * LD(2) ** -150
    assert (err <= tol).all(), float((err / tol).max())


# one workgroup for each 128 x 128, and workgroups of small pieces for few of them
@pytest.mark.parametrize("step", [65280, 16384])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_along_the_features(act, step):
    bits, x = _gates()
    for r in range(0, len(x), step):
        n = len(x[r:r + step])
        at = torch.arange(n, device=DEV)
        dh = torch.zeros((n, 128), dtype=torch.bfloat16, device=DEV)
        dh[at, at % 128] = 1
        gu = torch.ones((n, 256), dtype=torch.bfloat16, device=DEV)
        gu[at, at % 128] = to_dev_bf16(bits[r:r + step])
        _, s, _, _ = fq().gated_backward(dh, gu, act=act, tokens=False)
        a, da, ea, eda = _exact(act, x[r:r + step])
        _hold(s[0], da, eda)
        _hold(s[1], a, ea)


@pytest.mark.parametrize("step", [65280, 16384])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_along_the_tokens(act, step):
    bits, x = _gates()
    for r in range(0, len(x), step):
        n = len(x[r:r + step])
        dh = torch.ones((1, n), dtype=torch.bfloat16, device=DEV)
        gu = torch.ones((1, 2 * n), dtype=torch.bfloat16, device=DEV)
        gu[0, :n] = to_dev_bf16(bits[r:r + step])
        _, _, _, st = fq().gated_backward(dh, gu, act=act, rows=False)
        a, da, ea, eda = _exact(act, x[r:r + step])
        _hold(st[0, :n], da, eda)
        _hold(st[0, n:], a, ea)
