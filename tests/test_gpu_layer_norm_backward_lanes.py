"""Layer norm's backward pass of rows far from zero, whose mean times rstd FP32 cannot
hold: lanes past a row's end count for nothing."""

import numpy as np
import pytest

from gpu_util import fq
from oracle import training_step as ots
from test_gpu_layer_norm import U, _dev, _half, _num
from test_gpu_layer_norm_range import WIDTHS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x_dt,dy_dt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"),
                                        ("bf16", "f32")])
@pytest.mark.parametrize("N", WIDTHS)
def test_backward_of_rows_far_from_zero(N, x_dt, dy_dt):
    """x = mean, a power of two so large that mean * rstd overflows: z = 0, and the lanes
    past the row's end count for nothing."""
    rng = np.random.default_rng([N, 6])
    c = np.array([2.0 ** 126, -(2.0 ** 122), 2.0 ** 120, 1.0])
    M = len(c)
    x = _dev(np.broadcast_to(c[:, None], (M, N)), x_dt)
    dy = _dev(rng.standard_normal((M, N)) * 0.1, dy_dt)
    w = _dev(1 + 0.3 * rng.standard_normal(N))
    mean, rstd = _dev(c), _dev(np.full(M, 2.0 ** 9))
    dx, dw, db = fq().layer_norm_backward(dy, x, w, mean, rstd)
    DY, W = _num(dy), _num(w)
    rx, rw, rb = ots.layer_norm_backward(DY, _num(x), W, _num(mean), _num(rstd))
    gz = np.abs(DY * W)
    ex = 2.0 ** 9 * U * (6 * gz + 51 * gz.mean(axis=1, keepdims=True))
    assert np.all(np.abs(_num(dx) - rx) <= ex + _half(np.abs(rx) + ex, dx))
    assert not dw.any()
    assert np.all(np.abs(_num(db) - rb) <= 80 * U * np.abs(DY).sum(axis=0))
