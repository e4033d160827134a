"""Layer norm and its backward pass on the GPU against float64.

Tolerances (u = 2^-24; each FP32 operation is off by at most u of its result):
  mean   a sum of at most 16 terms in a lane, 6 steps over a wave and 16 over the
         waves, and a division: D = 40 u mean|x|.
  rstd   var about the computed mean is off by D^2 (exactly: the mean square about
         another point) and by the same sum's 38 u, 2 u of each square's own, and
         4 u of the quotient, eps and root's: relative 23 u + D^2 rstd^2 / 2.
  y      z is off by rstd D + (25 u + D^2 rstd^2 / 2) |z|; y = z w + b adds 2 u
         |z w| + u |y|; BF16 half an ulp (2^-8) of y and of y's own error.
  codes  half a step of E4M3 (2^-4 of the value, 2^-10 of the scale below the
         normals), y's error, and 3 u of the value for scale and multiplier.
         The scale is amax/448 of values within y's error.
  dx     z from the given mean and rstd 2 u |z|, gz = dy w 1 u, both row means 38 u
         + 6 u of the mean of magnitudes and 2 u of the division's; three
         products and differences: 5 u of each term's magnitude.
  dweight, dbias   a lane's sum over its rows (at most M/256 + 1 of them), at most
         16 over the lane groups of a workgroup, at most 1024/32 + 5 over workgroups:
         below (M/256 + 80) u of the sum of magnitudes, 3 u of each term's.
"""

import numpy as np
import pytest
import torch

from gpu_util import DEV, fq, host
from oracle import e4m3, quant as oquant, training_step as ots

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dev(a, dt="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(DT[dt])


def _num(t):
    return t.float().cpu().numpy().astype(np.float64)


def _rows(rng, M, N, dt, offset=0.5):
    x = rng.standard_normal((M, N)) * np.where(rng.random(N) < 0.02, 20.0, 1.0)
    return _dev(x + offset * rng.standard_normal((M, 1)), dt)


def _tolerance(x, w, b, eps):
    """(y, mean, rstd) in float64 and the FP32 error of each."""
    y, mean, rstd = ots.layer_norm(x, w, b, eps)
    D = 40 * U * np.abs(x).mean(axis=1)
    rel = 23 * U + 0.5 * (D * rstd) ** 2
    z = (x - mean[:, None]) * rstd[:, None]
    ez = (rstd * D)[:, None] + (2 * U + rel)[:, None] * np.abs(z)
    return (y, mean, rstd), (np.abs(w) * ez + 2 * U * np.abs(z * w) + U * np.abs(y), D, rstd * rel)


def _half(ref, t):
    return np.abs(ref) * 2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0


def _check_codes(q, s, y, ey, mode):
    """Codes and scales against y, which is off by at most ey."""
    M, N = y.shape
    g = lambda a: a.reshape(M, N // 128, 128)   # noqa: E731
    scale = _num(s).T
    amax, ea = np.abs(g(y)).max(axis=2), g(ey).max(axis=2)
    if mode == "f32":
        assert np.all(np.abs(scale - amax / 448) <= (ea + 3 * U * amax) / 448)
    else:
        # the least power of two that is enough for a value within the error
        up = lambda a: 2.0 ** np.ceil(np.log2(a / 448))   # noqa: E731
        assert np.all((scale >= up(amax - ea)) & (scale <= up(amax + ea)))
    wide = np.repeat(scale, 128, axis=1)
    v = e4m3.decode(host(q)) * wide
    assert np.all(np.abs(v - y) <= np.abs(y) * (2.0 ** -4 + 3 * U) + wide * 2.0 ** -10 + 1.1 * ey)


WIDTHS = [1, 2, 7, 8, 9, 63, 64, 65, 511, 512, 513, 1000, 1001, 1024, 1025, 2047, 2048, 2049, 4095,
          4096, 4097, 5000, 7168, 8191, 8192, 8193, 12001, 16383, 16384]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", WIDTHS)
def test_forward(N, dt):
    rng = np.random.default_rng([N, dt == "f32"])
    M = 5 if N > 600 else 11
    x = _rows(rng, M, N, dt)
    w, b = _dev(1 + 0.3 * rng.standard_normal(N)), _dev(rng.standard_normal(N))
    for bias in (b, None):
        for out in ("bf16", "f32"):
            y, mean, rstd = fq().layer_norm(x, w, bias, 1e-5, out_dtype=DT[out])
            (ry, rm, rr), (ey, em, er) = _tolerance(_num(x), _num(w),
                                                    None if bias is None else _num(bias), 1e-5)
            assert y.dtype == DT[out] and y.shape == (M, N)
            assert np.all(np.abs(_num(mean) - rm) <= em + 1e-45)
            assert np.all(np.abs(_num(rstd) - rr) <= er)
            assert np.all(np.abs(_num(y) - ry) <= ey + _half(np.abs(ry) + ey, y))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 5, 100, 128, 129, 200, 255, 256, 257])
def test_narrow_rows_that_share_a_wave(N, dt):
    """Every number of rows up to two workgroups' of the narrowest, each row as if alone."""
    rng = np.random.default_rng([N, 4])
    x, dy = _rows(rng, 33, N, dt), _rows(rng, 33, N, "bf16", 0)
    w, b = _dev(1 + 0.3 * rng.standard_normal(N)), _dev(rng.standard_normal(N))
    row = lambda t, i: t[i:i + 1].clone()   # noqa: E731  (a row's own start is not aligned)
    one = [fq().layer_norm(row(x, i), w, b, 1e-5) for i in range(33)]
    y, mean, rstd = (torch.cat([o[k] for o in one]) for k in range(3))
    dx = torch.cat([fq().layer_norm_backward(row(dy, i), row(x, i), w, *one[i][1:])[0]
                    for i in range(33)])
    for M in range(1, 34):
        ym, mm, rm = fq().layer_norm(x[:M], w, b, 1e-5)
        assert torch.equal(ym, y[:M]) and torch.equal(mm, mean[:M]) and torch.equal(rm, rstd[:M])
        dm = fq().layer_norm_backward(dy[:M], x[:M], w, mm, rm)
        assert torch.equal(dm[0], dx[:M])


@pytest.mark.parametrize("mode", ["f32", "pow2"])
@pytest.mark.parametrize("M,N", [(1, 128), (3, 256), (9, 512), (2, 640), (4, 1024), (130, 384),
                                 (5, 2048), (3, 4096), (1, 7168), (7, 7168), (2, 8192), (2, 16384)])
def test_forward_codes(M, N, mode):
    rng = np.random.default_rng([M, N])
    for dt in ("bf16", "f32"):
        x = _rows(rng, M, N, dt)
        w, b = _dev(1 + 0.3 * rng.standard_normal(N)), _dev(rng.standard_normal(N))
        q, s, mean, rstd, y = fq().layer_norm_quantized(x, w, b, 1e-6, mode, save_y=True,
                                                        out_dtype=torch.float32)
        (ry, rm, rr), (ey, em, er) = _tolerance(_num(x), _num(w), _num(b), 1e-6)
        assert np.all(np.abs(_num(y) - ry) <= ey)
        _check_codes(q, s, ry, ey, mode)
        # codes and y come from the same FP32 values: of y they are the quantizer's, bit for bit
        v = host(y)
        amax = np.abs(v.reshape(M, N // 128, 128)).max(axis=2)
        rule = oquant._scale_group_f32 if mode == "f32" else oquant._scale_group_pow2
        rq, rs = rule(v.reshape(M, N // 128, 128), amax[:, :, None])
        assert np.array_equal(host(q), np.asarray(rq).reshape(M, N))
        assert np.array_equal(host(s), np.asarray(rs).reshape(M, N // 128).T)
        # without y the codes are the same; a bare y too
        q2, s2, mean2, rstd2 = fq().layer_norm_quantized(x, w, b, 1e-6, mode)
        for a, c in ((q, q2), (s, s2), (mean, mean2), (rstd, rstd2)):
            assert torch.equal(a, c)
        assert torch.equal(fq().layer_norm(x, w, b, 1e-6, out_dtype=torch.float32)[0], y)


def test_forward_rows_that_are_constant_large_or_offset():
    """A constant row has z = 0 and y = bias; a row far from zero keeps its variance
    (taken about the mean); the largest finite values do not overflow."""
    N = 777
    rng = np.random.default_rng(4)
    w, b = _dev(1 + 0.3 * rng.standard_normal(N)), _dev(rng.standard_normal(N))
    x = rng.standard_normal((6, N)).astype(np.float32)
    x[0] = 0.0
    x[1] = 3.0
    x[2] += 4096.0
    x[3] *= 1e15
    x[4] *= 1e-20
    xd = _dev(x)
    y, mean, rstd = fq().layer_norm(xd, w, b, 1e-5, out_dtype=torch.float32)
    (ry, rm, rr), (ey, em, er) = _tolerance(x.astype(np.float64), _num(w), _num(b), 1e-5)
    assert torch.equal(y[0], b) and torch.equal(y[1], b)
    assert np.all(np.abs(_num(mean) - rm) <= em)
    assert np.all(np.abs(_num(rstd) - rr) <= er) and np.all(np.abs(_num(y) - ry) <= ey)


@pytest.mark.parametrize("x_dt,dy_dt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"),
                                        ("bf16", "f32")])
@pytest.mark.parametrize("M,N", [(1, 1), (3, 7), (1, 64), (2, 65), (300, 8), (5, 511), (1025, 512),
                                 (7, 513), (1100, 130), (9, 1001), (6, 1024), (5, 1025), (3, 2048),
                                 (4, 2049), (300, 3000), (5, 4096), (3, 4097), (260, 7168),
                                 (2, 8192), (3, 8193), (2, 12001), (2, 16384)])
def test_backward(M, N, x_dt, dy_dt):
    rng = np.random.default_rng([M, N])
    x = _rows(rng, M, N, x_dt)
    dy = _dev(rng.standard_normal((M, N)) * 0.1, dy_dt)
    w = _dev(1 + 0.3 * rng.standard_normal(N))
    _, mean, rstd = fq().layer_norm(x, w, None, 1e-5)
    dx, dw, db = fq().layer_norm_backward(dy, x, w, mean, rstd)
    X, DY, W, R = _num(x), _num(dy), _num(w), _num(rstd)[:, None]
    rx, rw, rb = ots.layer_norm_backward(DY, X, W, _num(mean), _num(rstd))
    z = np.abs((X - _num(mean)[:, None]) * R)
    gz = np.abs(DY * W)
    m2, m1 = gz.mean(axis=1, keepdims=True), (gz * z).mean(axis=1, keepdims=True)
    ex = R * U * (6 * gz + 51 * m2 + 53 * z * m1)
    assert dx.dtype == x.dtype
    assert np.all(np.abs(_num(dx) - rx) <= ex + _half(np.abs(rx) + ex, dx))
    adds = M / 256 + 80
    assert np.all(np.abs(_num(dw) - rw) <= (adds + 3) * U * (np.abs(DY) * z).sum(axis=0))
    assert np.all(np.abs(_num(db) - rb) <= adds * U * np.abs(DY).sum(axis=0))
    # no dbias, and the same bits again
    dx2, dw2, none = fq().layer_norm_backward(dy, x, w, mean, rstd, bias=False)
    assert none is None and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_backward_against_differences():
    """sum(dy y(x + h d)) along random directions d, y from the forward call in FP32.
    With values of order 1 and N terms the two sums carry about sqrt(N) u each of
    rounding, 2 sqrt(N) u / 2h of the difference's; third order h^2/6: at h = 2^-6
    1e-4 and 1e-4 of sqrt(N)."""
    rng = np.random.default_rng(8)
    M, N, h = 6, 640, 2.0 ** -6
    x, dy = rng.standard_normal((M, N)), _dev(rng.standard_normal((M, N)))
    w = _dev(1 + 0.3 * rng.standard_normal(N))
    xd = _dev(x)
    _, mean, rstd = fq().layer_norm(xd, w, None, 1e-5, out_dtype=torch.float32)
    dx, dw, db = fq().layer_norm_backward(dy, xd, w, mean, rstd)
    for _ in range(5):
        d = rng.standard_normal((M, N))
        d /= np.linalg.norm(d)

        def loss(t):
            y = fq().layer_norm(_dev(_num(xd) + t * d), w, None, 1e-5, out_dtype=torch.float32)[0]
            return float((y.double() * dy.double()).sum())
        want = float((dx.double() * torch.from_numpy(d).to(DEV)).sum())
        assert abs((loss(h) - loss(-h)) / (2 * h) - want) < 2e-4 * np.sqrt(M * N)


def test_no_rows():
    w, b = torch.ones(200, device=DEV), torch.ones(200, device=DEV)
    x = torch.empty((0, 200), device=DEV)
    y, mean, rstd = fq().layer_norm(x, w, b)
    assert y.shape == (0, 200) and mean.shape == rstd.shape == (0,)
    dx, dw, db = fq().layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 200) and not dw.any() and not db.any()


def test_rows_past_32_bit_offsets():
    """Rows whose bytes begin past 2^32: the last ones as a call of their own."""
    N = 16384
    M = (1 << 32) // (2 * N) + 3
    x = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    x[-4:] = torch.randn((4, N), device=DEV).to(torch.bfloat16)
    w, b = torch.rand(N, device=DEV) + 0.5, torch.rand(N, device=DEV)
    q, s, mean, rstd, y = fq().layer_norm_quantized(x, w, b, save_y=True)
    tail = fq().layer_norm_quantized(x[-4:], w, b, save_y=True)
    assert torch.equal(q[-4:], tail[0]) and torch.equal(s[:, -4:], tail[1])
    assert torch.equal(y[-4:], tail[4]) and torch.equal(mean[-4:], tail[2])
    dx, dw, db = fq().layer_norm_backward(y, x, w, mean, rstd)
    want = fq().layer_norm_backward(y[-4:], x[-4:], w, mean[-4:], rstd[-4:])
    assert torch.equal(dx[-4:], want[0])
