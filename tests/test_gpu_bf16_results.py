"""BF16 results of layer norm and AdamW are torch's rounding of the FP32 values, bit for
bit, and NaN for every NaN, whatever its bits."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, fq, host

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
NANS = [0x7FC00000, 0xFFC00000, 0x7FFFFFFF, 0xFFFFFFFF, 0x7FFF8001, 0xFFFF8000, 0x7F800001]


def _bits(values):
    return torch.from_numpy(np.array(values, dtype=np.uint32).view(np.float32)).to(DEV)


def _spread(n):
    """Every exponent, subnormals among them, ties and their neighbours."""
    rng = np.random.default_rng(1)
    low = rng.choice([0x7FFF, 0x8000, 0x8001, 0x0000, 0xFFFF, 0x1234], n).astype(np.uint32)
    high = rng.integers(0, 0x7F80, n).astype(np.uint32) | rng.choice([0, 0x8000], n).astype(np.uint32)
    return _bits((high << 16) | low)


@pytest.mark.parametrize("n", [4096, 4101])
@pytest.mark.parametrize("eight", [False, True])
def test_copies_of_parameters(eight, n):
    """lr = 0 and no gradient: the parameter stays as it is."""
    p = _spread(n)
    p[:len(NANS)] = _bits(NANS)
    p[-len(NANS):] = _bits(NANS)
    was, copy = p.clone(), torch.zeros(n, dtype=BF16, device=DEV)
    g = torch.zeros(n, device=DEV)
    if eight:
        u8 = [torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
        sc = [torch.zeros(-(-n // 128), device=DEV) for _ in range(2)]
        fq().adamw_8bit([p], [g], [u8[0]], [sc[0]], [u8[1]], [sc[1]], 1, lr=0.0, copies=[copy])
    else:
        m = [torch.zeros(n, device=DEV) for _ in range(2)]
        fq().adamw([p], [g], [m[0]], [m[1]], 1, lr=0.0, copies=[copy])
    nan = torch.isnan(was)
    assert torch.equal(p[~nan].view(torch.int32), was[~nan].view(torch.int32))
    assert torch.isnan(p[nan]).all() and torch.isnan(copy[nan].float()).all()
    want = was[~nan].cpu().to(BF16)
    assert torch.equal(copy[~nan].cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("N", [100, 101, 512, 7168])
def test_rows_of_nan(N):
    """Whatever its bits, a NaN in a row is NaN in all of y and of dx."""
    w = torch.ones(N, device=DEV)
    for x_type in (torch.float32, BF16):
        x = torch.randn((len(NANS), N), device=DEV)
        x[:, N // 2] = _bits(NANS)
        x = x.to(x_type)
        x[:, N // 2] = float("nan")
        if x_type == torch.float32:
            x[:, N // 2] = _bits(NANS)
        else:
            x[-1, N // 2:N // 2 + 1].view(torch.int16).fill_(-1)      # 0xFFFF
        y, mean, rstd = fq().layer_norm(x, w)
        assert torch.isnan(y.float()).all()
        dx, _, _ = fq().layer_norm_backward(x, x, w, mean, rstd)
        assert torch.isnan(dx.float()).all()
        z = torch.randn((len(NANS), N), device=DEV).to(BF16)
        _, mean, rstd = fq().layer_norm(z, w)
        dx, _, _ = fq().layer_norm_backward(x, z, w, mean, rstd)
        assert torch.isnan(dx.float()).all()


def test_layer_norm_rounds_as_torch_does():
    """y in BF16 is y in FP32 rounded, over many exponents (the weight's)."""
    N = 4096
    x = torch.randn((6, N), device=DEV)
    w = _spread(N)
    w = torch.where(w.abs() < 1e37, w, 1.0)
    y32 = fq().layer_norm(x, w, out_dtype=torch.float32)[0]
    y16 = fq().layer_norm(x, w)[0]
    assert np.array_equal(host(y16.view(torch.int16)), host(y32.cpu().to(BF16).view(torch.int16)))
