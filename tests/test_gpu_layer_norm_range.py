"""Layer norm over the range of FP32: rows whose squares overflow or underflow, sums past
the largest value, eps = 0.  Tolerances are those of the other rows (of values of order
1); what scaling by powers of two adds is below them: an element of a large row loses
what is below 2^-49, 2^-109 of the 2^60 at least that such a row deviates."""

import numpy as np
import pytest
import torch

from gpu_util import fq, host
from oracle import training_step as ots
from test_gpu_layer_norm import DT, U, _check_codes, _dev, _half, _num, _tolerance

pytestmark = pytest.mark.gpu
WIDTHS = [1, 77, 128, 200, 256, 400, 512, 777, 1024, 2000, 2048, 4096, 5000, 7168, 8192, 9001, 16384]
SCALES = [1e-37, 1e-33, 1e-28, 1e-24, 1e-20, 1e-16, 1e-14, 1e-10, 1e15, 1e17, 1e18, 1e19, 1e20,
          1e25, 1e30, 1e35, 3e36]


def _rows(rng, N, dt):
    """A row of each scale about zero, then of each far from it, in no order."""
    z = rng.standard_normal((2 * len(SCALES), N))
    s = np.array(SCALES * 2)[:, None]
    x = s * z
    x[len(SCALES):] += 3 * s[len(SCALES):]
    return _dev(x[rng.permutation(len(x))], dt)


@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-5])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [n for n in WIDTHS if n > 1])
def test_forward(N, dt, eps):
    rng = np.random.default_rng([N, dt == "f32", 5])
    x = _rows(rng, N, dt)
    w, b = _dev(1 + 0.3 * rng.standard_normal(N)), _dev(rng.standard_normal(N))
    (ry, rm, rr), (ey, em, er) = _tolerance(_num(x), _num(w), _num(b), float(np.float32(eps)))
    for out in ("bf16", "f32"):
        y, mean, rstd = fq().layer_norm(x, w, b, eps, out_dtype=DT[out])
        assert np.all(np.abs(_num(mean) - rm) <= em + 1e-45)
        assert np.all(np.abs(_num(rstd) - rr) <= er)
        assert np.all(np.abs(_num(y) - ry) <= ey + _half(np.abs(ry) + ey, y))
    if N % 128 == 0:
        for mode in ("f32", "pow2"):
            q, s, mean2, rstd2 = fq().layer_norm_quantized(x, w, b, eps, mode)
            assert torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
            _check_codes(q, s, ry, ey, mode)


@pytest.mark.parametrize("N", WIDTHS)
def test_constant_rows(N):
    """Equal values: z = 0 and y = bias, rstd = 1/sqrt(eps), where their sum is exact
    (a value of few bits); 2^126 and a sum of them past the largest value too."""
    c = np.array([0.0, 2.0 ** -130, 2.0 ** -60, 3.0, 2.0 ** 70, -(2.0 ** 100), 2.0 ** 126])
    x = _dev(np.broadcast_to(c[:, None], (len(c), N)))
    w, b = _dev(np.full(N, 1.25)), _dev(np.linspace(-1, 1, N))
    for eps in (1e-5, 1e-12, 1e-36):
        y, mean, rstd = fq().layer_norm(x, w, b, eps, out_dtype=torch.float32)
        assert torch.equal(mean, x[:, 0])
        assert torch.equal(y, b.expand(len(c), N))
        want = 1 / np.sqrt(float(np.float32(eps)))
        assert np.all(np.abs(_num(rstd) - want) <= 23 * U * want)


def test_rows_that_are_not_finite_are_lost_alone():
    """A NaN or an infinity: the row's y is NaN throughout or its formula's, and the rows
    beside it, of the same wave or workgroup, are as without it."""
    for N in (100, 256, 512, 1000, 7168):
        rng = np.random.default_rng(N)
        x = _dev(rng.standard_normal((9, N)))
        w, b = _dev(1 + 0.3 * rng.standard_normal(N)), _dev(rng.standard_normal(N))
        want = fq().layer_norm(x, w, b)
        x[2, 5], x[4, N - 1], x[7, 0] = float("nan"), float("inf"), -float("inf")
        got = fq().layer_norm(x, w, b)
        keep = [0, 1, 3, 5, 6, 8]
        for g, o in zip(got, want):
            assert torch.equal(g[keep], o[keep])
        assert torch.isnan(got[0][[2, 4, 7]].float()).all()


def test_backward_over_the_range_of_scales():
    """The gradients of the forward's rows, from its mean and rstd."""
    for N in (200, 777, 2048, 7168):
        rng = np.random.default_rng([N, 7])
        s = np.array([1e-30, 1e-20, 1e18, 1e20, 1e30])[:, None]
        x = _dev(s * rng.standard_normal((5, N)))
        dy = _dev(s * rng.standard_normal((5, N)) * 0.1)
        w = _dev(1 + 0.3 * rng.standard_normal(N))
        _, mean, rstd = fq().layer_norm(x, w, None, 0.0)
        dx, _, _ = fq().layer_norm_backward(dy, x, w, mean, rstd)
        X, DY, W, R = _num(x), _num(dy), _num(w), _num(rstd)[:, None]
        rx, _, _ = ots.layer_norm_backward(DY, X, W, _num(mean), _num(rstd))
        z, gz = np.abs((X - _num(mean)[:, None]) * R), np.abs(DY * W)
        m2, m1 = gz.mean(axis=1, keepdims=True), (gz * z).mean(axis=1, keepdims=True)
        assert np.all(np.abs(_num(dx) - rx) <= R * U * (6 * gz + 51 * m2 + 53 * z * m1))
        assert np.isfinite(host(rstd)).all()
