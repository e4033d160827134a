"""The 8-bit feed-forward calls on the GPU against oracle.feed_forward.

Tolerances (u = 2^-24):
  quantize_token_i8  bit for bit.
  gemm_i8            the integer sum is exact; its conversion and two products
                     (and one sum) round once each: 4u (|C - b| + |b|), and half
                     a BF16 ulp for BF16 output.
  act(x) = x sigma(y)  exp(-y) is off by the rounding of y (a few u of |y|,
                     multiplied by log2 e) and the exponential's own ulp, the
                     rest by an ulp each: u (16 + 8 |y|) relative.
  gated              with gate off by eg and up by eu: |act'| < 1.2, so
                     1.2 eg (|up| + eu) + |act(gate)| eu + (act's own + 2u) |h|.
  gated_backward     dY carries three factors of a few u: e = u (16 + 8 |y|)
                     |dh| (|up| (1 + |x| |y'|) or |gate|), on which its scale
                     (relative to the group's largest) and its codes (half a
                     step of E4M3 at the value, plus e) are held.
"""

import numpy as np
import pytest
import torch

import workloads
from gpu_util import DEV, bf16_to_bits, fq, host, to_dev_bf16
from oracle import e4m3, feed_forward as off, gemm as ogemm, mfma_model, quant as oquant

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _bf16(x):
    """float array -> (its BF16 rounding as float32, device tensor)."""
    bits = workloads.bf16_bits(np.asarray(x, dtype=np.float32))
    return oquant.bf16_bits_to_f32(bits), to_dev_bf16(bits)


def _f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV)


def _i8(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int8)).to(DEV)


def _value(t):
    return t.float().cpu().numpy().astype(np.float64)


def _half(ref, t):
    return ogemm.bf16_half_ulp(ref) * (1 + 2.0 ** -6) if t.dtype == torch.bfloat16 else 0.0


def _act_err(act, x):
    return U * (16 + 8 * np.abs(off.act_arg(act, x)))


# --------------------------------------------------------------- quantize_token_i8
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 16), (2, 511), (2, 512), (7, 513), (4, 1025),
                                 (3, 2047), (4, 2049), (2, 4097), (2, 8192), (2, 8193), (2, 16385),
                                 (1, 40000), (130, 257)])
def test_quantize_token_i8(M, K):
    rng = np.random.default_rng([M, K])
    x = rng.standard_normal((M, K)) * np.exp(rng.uniform(-3, 3, (M, 1)))
    x[:, ::3] = x[:, :1] / 2          # halves of a value: ties where it is the largest
    if M > 1:
        x[1] = 0                      # flushed
    if M > 2:
        x[2] *= 2.0 ** -140           # 1/amax overflows: flushed, or subnormal values
    if M > 3:
        x[3, -1] = 3.3e38
    xf, xd = _bf16(x)
    q, s = fq().quantize_token_i8(xd)
    rq, rs = off.quantize_token_i8(xf)
    assert q.shape == rq.shape
    assert np.array_equal(host(q), rq)
    assert np.array_equal(host(s).view(np.uint32), rs.view(np.uint32))


# ------------------------------------------------------------------------ gemm_i8
def _i8_operands(rng, M, N, K, extreme=False):
    if extreme:
        qa = np.where(rng.random((M, K)) < 0.5, -128, 127).astype(np.int8)
        qw = np.where(rng.random((N, K)) < 0.5, -128, 127).astype(np.int8)
        qa[0], qw[0] = -128, -128     # the largest sum there is
    else:
        qa = rng.integers(-127, 128, (M, K)).astype(np.int8)
        qw = rng.integers(-127, 128, (N, K)).astype(np.int8)
    sa = rng.uniform(0.001, 0.1, M).astype(np.float32)
    sw = rng.uniform(1e-4, 1e-3, N).astype(np.float32)
    return qa, sa, qw, sw


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 5, 48), (2, 16, 128), (15, 17, 144), (16, 128, 1040),
                                   (17, 33, 2048), (31, 64, 272), (33, 127, 512), (64, 200, 1024),
                                   (65, 129, 656), (128, 128, 128), (130, 257, 1008),
                                   (257, 300, 400), (300, 513, 2064), (600, 1030, 336),
                                   (1025, 260, 64)])
def test_gemm_i8(M, N, K, out):
    rng = np.random.default_rng([M, N, K])
    qa, sa, qw, sw = _i8_operands(rng, M, N, K)
    bias = rng.standard_normal(N).astype(np.float32) if (M + N) % 2 else None
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    c = fq().gemm_i8(_i8(qa), _f32(sa), _i8(qw), _f32(sw), out_dtype=dt,
                     bias=None if bias is None else _f32(bias))
    ref = off.gemm_i8(qa, sa, qw, sw)
    b = 0.0 if bias is None else bias.astype(np.float64)[None, :]
    tol = 4 * U * (np.abs(ref) + np.abs(b))
    ref = ref + b
    assert np.all(np.abs(_value(c) - ref) <= tol + _half(ref, c))


def test_gemm_i8_largest_sum():
    """K = 131056, every code -128: the sum is 2^31 - 2^18, still an int32."""
    rng = np.random.default_rng(5)
    for M, N in ((3, 20), (200, 140)):
        qa, sa, qw, sw = _i8_operands(rng, M, N, 131056, extreme=True)
        c = fq().gemm_i8(_i8(qa), _f32(sa), _i8(qw), _f32(sw))
        ref = off.gemm_i8(qa, sa, qw, sw)
        assert ref[0, 0] > 0
        assert np.all(np.abs(_value(c) - ref) <= 4 * U * np.abs(ref))


def test_gemm_i8_empty():
    f = fq()
    z = torch.empty((0, 32), dtype=torch.int8, device=DEV)
    w, ws = _i8(np.ones((5, 32))), _f32(np.ones(5))
    assert f.gemm_i8(z, _f32(np.ones(0)), w, ws).shape == (0, 5)
    with pytest.raises(f.Fp8qError):
        f.gemm_i8(torch.empty((4, 0), dtype=torch.int8, device=DEV), _f32(np.ones(4)),
                  torch.empty((5, 0), dtype=torch.int8, device=DEV), ws)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", [(1, 1, 16), (1, 100, 512), (9, 7, 144), (16, 64, 2048),
                                   (20, 130, 272), (64, 33, 400), (65, 128, 656), (130, 65, 1008),
                                   (257, 128, 256), (300, 257, 400), (700, 520, 336)])
def test_gemm_i8_gated(M, F, K, act):
    rng = np.random.default_rng([M, F, K])
    qa, sa, qw, sw = _i8_operands(rng, M, 2 * F, K)
    sw[:F] *= 4
    if M > 4:
        sa[3] *= 200                  # gates far out on both sides
    Y = off.gemm_i8(qa, sa, qw, sw)
    ref = off.gated(act, Y)
    eg, eu = 4 * U * np.abs(Y[:, :F]), 4 * U * np.abs(Y[:, F:])
    tol = (1.2 * eg * (np.abs(Y[:, F:]) + eu) + np.abs(off.act(act, Y[:, :F])) * eu
           + (_act_err(act, Y[:, :F]) + 2 * U) * np.abs(ref) + 1e-36)
    for dt in (torch.float32, torch.bfloat16):
        h = fq().gemm_i8_gated(_i8(qa), _f32(sa), _i8(qw), _f32(sw), act=act, out_dtype=dt)
        assert np.all(np.abs(_value(h) - ref) <= tol + _half(ref, h))


# ------------------------------------------------------------- gated, E4M3 operands
def _e4m3_operands(rng, M, N, K, outliers=False):
    a = rng.standard_normal((M, K)).astype(np.float32)
    if outliers:
        a[:, rng.integers(0, K, 2)] *= 50
    w = (rng.standard_normal((N, K)) * 2.5 / np.sqrt(K)).astype(np.float32)
    qa, sa = oquant.quantize_act(workloads.bf16_bits(a))
    qw, sw = oquant.quantize_weight(workloads.bf16_bits(w))
    return qa, sa, qw, sw


def _u8(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _check_gated(act, h, gu, qa, sa, qw, sw):
    F = qw.shape[0] // 2
    Y = ogemm.gemm(qa, sa, qw, sw)
    G = qa.shape[1] // 128
    # the bound of the FP8 matrix core's product, for any order of its chunks
    e = mfma_model.truncation_bound(qa, sa, qw, sw) + (G + 20) * U * ogemm.abs_bound(qa, sa, qw, sw)
    if gu is not None:
        assert np.all(np.abs(_value(gu) - Y) <= e + _half(Y, gu))
    g, u, eg, eu = Y[:, :F], Y[:, F:], e[:, :F], e[:, F:]
    ref = off.gated(act, Y)
    tol = 1.2 * eg * (np.abs(u) + eu) + np.abs(off.act(act, g)) * eu \
        + (_act_err(act, g) + 2 * U) * np.abs(ref) + 1e-36
    assert np.all(np.abs(_value(h) - ref) <= tol + _half(ref, h))


@pytest.mark.parametrize("M,F,K,act,save", [
    (1, 128, 128, "silu", False), (1, 256, 1152, "gelu_tanh", True), (7, 128, 512, "silu", True),
    (16, 128, 1024, "silu", False), (17, 256, 256, "gelu_tanh", True), (48, 128, 640, "silu", True),
    (64, 384, 384, "silu", False), (65, 128, 256, "gelu_tanh", True), (129, 256, 512, "silu", True),
    (200, 384, 256, "silu", False), (257, 128, 384, "silu", True), (300, 512, 256, "gelu_tanh", True),
    (520, 640, 128, "silu", True)])
def test_gemm_gated(M, F, K, act, save):
    rng = np.random.default_rng([M, F, K])
    qa, sa, qw, sw = _e4m3_operands(rng, M, 2 * F, K, outliers=M % 2 == 1)
    for dt in (torch.bfloat16, torch.float32):
        r = fq().gemm_gated(_u8(qa), _u8(sa), _u8(qw), _u8(sw), act=act, out_dtype=dt,
                            save_gate_up=save)
        h, gu = r if save else (r, None)
        assert h.dtype == dt
        _check_gated(act, h, gu, qa, sa, qw, sw)


@pytest.mark.parametrize("counts,F,K,act", [
    ([0, 5, 0, 1, 64, 0], 128, 256, "silu"), ([65, 3, 130], 256, 384, "gelu_tanh"),
    ([0, 0, 0], 128, 128, "silu"), ([300], 128, 256, "silu"), ([1] * 70, 128, 128, "silu"),
    ([17, 200, 150, 0, 257, 90], 384, 256, "silu")])
def test_grouped_gemm_gated(counts, F, K, act):
    f = fq()
    rng = np.random.default_rng(len(counts) + F + K)
    G, spare = len(counts), 9         # rows past off[G] stay as they are
    ends = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(ends[-1]) + spare
    qa, sa, qw, sw = _e4m3_operands(rng, M, G * 2 * F, K)
    qw3, sw3 = qw.reshape(G, 2 * F, K), sw.reshape(G, 2 * F // 128, K // 128)
    h = torch.full((M, F), 7.0, dtype=torch.bfloat16, device=DEV)
    gu = torch.full((M, 2 * F), 7.0, dtype=torch.bfloat16, device=DEV)
    f.fp8q_grouped_gemm_gated(_u8(qa), _u8(sa), _u8(ends), _u8(qw3), _u8(sw3), h, act, gu)
    assert (h[ends[-1]:] == 7).all() and (gu[ends[-1]:] == 7).all()
    for e in range(G):
        lo, hi = ends[e], ends[e + 1]
        if hi > lo:
            _check_gated(act, h[lo:hi], gu[lo:hi], qa[lo:hi], sa[:, lo:hi], qw3[e], sw3[e])


@pytest.mark.parametrize("ends", [[1, 4, 9], [0, 6, 4], [0, 4, 41], [0, -3, 9]])
def test_grouped_gemm_gated_invalid_offsets_write_nothing(ends):
    f = fq()
    rng = np.random.default_rng(1)
    qa, sa, qw, sw = _e4m3_operands(rng, 40, 2 * 256, 128)
    h = torch.full((40, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    f.fp8q_grouped_gemm_gated(_u8(qa), _u8(sa), _u8(np.array(ends, dtype=np.int32)),
                              _u8(qw.reshape(2, 256, 128)), _u8(sw.reshape(2, 2, 1)), h)
    assert (h == 7).all()


# ------------------------------------------------------------------ gated_backward
def _half_step(v):
    """Half the spacing of E4M3 values at |v| <= 448 (coarser of the two sides)."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    return 2.0 ** (e - 4)


def _check_codes(q, s, ref, err, mode):
    """q: codes [R][n], s: scales [n/128][R], of ref [R][n] known within err."""
    R, n = ref.shape
    sc = s.T.astype(np.float64)                           # [R][n/128]
    grp = np.abs(ref).reshape(R, n // 128, 128)
    top, etop = grp.max(axis=2), err.reshape(R, n // 128, 128).max(axis=2)
    if mode == "f32":
        assert np.all(np.abs(sc - top / 448) <= etop / 448 + 2 * U * top / 448 + 2.0 ** -148)
    else:
        live = top > etop                 # a group within its error of zero may be flushed
        assert np.all(sc[top == 0] == 0)
        assert np.all(np.log2(sc[live]) % 1 == 0)
        assert np.all(448 * sc[live] >= (top - etop)[live])
        assert np.all(224 * sc[live] < (top + etop)[live])
    wide = np.repeat(sc, 128, axis=1)
    v = e4m3.decode(q) * wide
    # half a step at the value, at most one rounding of the product before it
    with np.errstate(divide="ignore", invalid="ignore"):
        step = np.where(wide > 0, _half_step(ref / np.where(wide > 0, wide, 1)) * wide, 0)
    assert np.all(np.abs(v - ref) <= step * (1 + 1e-6) + 2 * err + 4 * U * np.abs(ref))


@pytest.mark.parametrize("mode", ["f32", "pow2"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F", [(1, 128), (5, 256), (127, 128), (128, 128), (129, 384), (300, 256)])
def test_gated_backward(M, F, act, mode):
    rng = np.random.default_rng([M, F])
    dh = rng.standard_normal((M, F)) * 0.01
    Y = rng.standard_normal((M, 2 * F)) * 2
    if M > 4:
        dh[3] = 0                                         # a row without gradient
        Y[:, 5] = np.where(np.arange(M) % 2, 200.0, -200.0)   # saturated gates
        Y[:, 6] = np.where(np.arange(M) % 2, 3e38, -3e38)
        Y[:, F + 6] = 1e-30
        dh[:, 6] = 1e-3
    if M > 200:
        dh[:, 70] = 0                                     # a feature without gradient
    dhf, dhd = _bf16(dh)
    Yf, Yd = _bf16(Y)
    with np.errstate(over="ignore", invalid="ignore"):
        g, u = Yf[:, :F].astype(np.float64), Yf[:, F:].astype(np.float64)
        gc = np.clip(g, -1e3, 1e3)
        y = off.act_arg(act, gc)
        dy = 1.0 if act == "silu" else 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * gc ** 2)
        big = np.abs(g) > 1e3                             # act is x or 0 there, exactly
        a = np.where(big, np.maximum(g, 0), off.act(act, gc))
        da = np.where(big, g > 0, off.act_grad(act, gc))
        rel = U * (16 + 8 * np.minimum(np.abs(y), 100))
        ref = np.concatenate([dhf * u * da, dhf * a], axis=1)
        err = np.concatenate([rel * np.abs(dhf * u) * (np.abs(da) + np.where(
            big, 0, np.abs(gc * dy) * off._sigma(y) * off._sigma(-y))), rel * np.abs(dhf * a)], axis=1)
    assert np.all(np.isfinite(ref))
    err += 1e-36
    q, s, qt, st = fq().gated_backward(dhd, Yd, act=act, mode=mode)
    _check_codes(host(q), host(s), ref, err, mode)
    Mp = -(-M // 128) * 128
    pad = lambda v: np.concatenate([v, np.zeros((Mp - M, 2 * F))]).T   # noqa: E731
    assert qt.shape == (2 * F, Mp) and not host(qt)[:, M:].any()
    _check_codes(host(qt), host(st), pad(ref), pad(err), mode)
    # either pair alone is the same pair
    q1, s1, n1, n2 = fq().gated_backward(dhd, Yd, act=act, mode=mode, tokens=False)
    n3, n4, qt1, st1 = fq().gated_backward(dhd, Yd, act=act, mode=mode, rows=False)
    assert n1 is n2 is n3 is n4 is None
    assert torch.equal(q1, q) and torch.equal(s1, s) and torch.equal(qt1, qt) and torch.equal(st1, st)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("mode", ["f32", "pow2"])
@pytest.mark.parametrize("M,part", [(1200, 128), (1200, 384), (1150, 1100)])
def test_gated_backward_of_a_part_is_the_part_of_it(M, part, act, mode):
    """Few and many groups (kernels of their own) agree bit for bit: a call on
    the first tokens gives the first rows and groups of the whole one."""
    F = 2048
    g = torch.Generator(device=DEV)
    g.manual_seed(M + part)
    dh = torch.randn(M, F, generator=g, device=DEV).to(torch.bfloat16)
    Y = (2 * torch.randn(M, 2 * F, generator=g, device=DEV)).to(torch.bfloat16)
    q, s, qt, st = fq().gated_backward(dh, Y, act=act, mode=mode)
    for n in range(0, part, part if part < 1000 else 128):
        m = min(n + (part if part < 1000 else 128), M)
        q1, s1, qt1, st1 = fq().gated_backward(dh[n:m], Y[n:m], act=act, mode=mode)
        assert torch.equal(q1, q[n:m]) and torch.equal(s1, s[:, n:m])
        assert torch.equal(qt1, qt[:, n:n + qt1.shape[1]])
        assert torch.equal(st1, st[n // 128:n // 128 + st1.shape[0]])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_backward_against_differences(act):
    """The dequantized dY against central differences of the forward formula:
    codes are within 2^-4 of the value, or 2^-10 of the group's scale's 448."""
    rng = np.random.default_rng(11)
    M, F = 4, 128
    dhf, dhd = _bf16(rng.standard_normal((M, F)))
    Yf, Yd = _bf16(rng.standard_normal((M, 2 * F)) * 2)
    q, s, _, _ = fq().gated_backward(dhd, Yd, act=act, tokens=False)
    got = e4m3.decode(host(q)) * np.repeat(host(s).T.astype(np.float64), 128, axis=1)
    h = 1e-5
    Y, dh = Yf.astype(np.float64), dhf.astype(np.float64)
    up, dn = Y.copy(), Y.copy()
    up[:, :F] += h
    dn[:, :F] -= h
    dg = dh * (off.gated(act, up) - off.gated(act, dn)) / (2 * h)
    up, dn = Y.copy(), Y.copy()
    up[:, F:] += h
    dn[:, F:] -= h
    du = dh * (off.gated(act, up) - off.gated(act, dn)) / (2 * h)
    ref = np.concatenate([dg, du], axis=1)
    wide = np.repeat(host(s).T.astype(np.float64), 128, axis=1)
    assert np.all(np.abs(got - ref) <= np.abs(ref) * 2.0 ** -4 + wide * 2.0 ** -10 + 1e-7)


# ----------------------------------------------------------- streams, graphs, layers
def _layer_inputs(seed, M=200, F=256, K=512):
    rng = np.random.default_rng(seed)
    f = fq()
    _, x = _bf16(rng.standard_normal((M, K)))
    _, w = _bf16(rng.standard_normal((2 * F, K)) * 0.1)
    _, dh = _bf16(rng.standard_normal((M, F)) * 0.01)
    return f, x, w, dh


def _layer(f, x, w8, wq, ws, dh):
    xq, xs = f.quantize_token_i8(x)
    y = f.gemm_i8(xq, xs, *w8, out_dtype=torch.bfloat16)
    h8 = f.gemm_i8_gated(xq, xs, *w8)
    aq, as_ = f.quantize_act(x)
    h, gu = f.gemm_gated(aq, as_, wq, ws, save_gate_up=True)
    return [xq, xs, y, h8, h, gu, *f.gated_backward(dh, gu)]


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_calls_run_on_the_current_stream():
    f, x, w, dh = _layer_inputs(1)
    w8, (wq, ws) = f.quantize_token_i8(w), f.quantize_weight(w)
    ref = _layer(f, x, w8, wq, ws, dh)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        x2 = torch.empty_like(x)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            x2.copy_(x)               # ordered before the layer by the stream alone
            got = _layer(f, x2, w8, wq, ws, dh)
        torch.cuda.current_stream().wait_stream(side)
        assert _same(got, ref)


def test_graph_replays_match_eager():
    f, x, w, dh = _layer_inputs(2)
    w8, (wq, ws) = f.quantize_token_i8(w), f.quantize_weight(w)
    _layer(f, x, w8, wq, ws, dh)
    torch.cuda.synchronize()
    buf = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _layer(f, buf, w8, wq, ws, dh)
    for k in range(4):
        _, xk = _bf16(np.random.default_rng(100 + k).standard_normal(tuple(x.shape)))
        ref = _layer(f, xk, w8, wq, ws, dh)
        torch.cuda.synchronize()
        buf.copy_(xk)
        g.replay()
        torch.cuda.synchronize()
        assert _same(out, ref)


@pytest.mark.parametrize("M", [256, 200])
def test_training_step_gradients(M):
    """Forward, backward and both gradient GEMMs of the gate/up projection: dX
    and dW against float64 products of the operands the calls hand over."""
    f, x, w, dh = _layer_inputs(3, M=M)
    K = x.shape[1]
    aq, as_ = f.quantize_act(x)
    wq, ws = f.quantize_weight(w)
    h, gu = f.gemm_gated(aq, as_, wq, ws, save_gate_up=True)
    q, s, qt, st = f.gated_backward(dh, gu)
    wt, wts = f.quantize_weight_t(w)
    dx = f.gemm(q, s, wt, wts, precise=True)
    pad = -M % 128
    xt, xts = f.quantize_act_t(torch.nn.functional.pad(x, (0, 0, 0, pad)))
    dw = f.gemm_rowscaled(qt, st, xt, xts, precise=True)
    assert dx.shape == (M, K) and dw.shape == w.shape
    H = lambda t: host(t)   # noqa: E731
    assert np.all(np.abs(_value(dx) - ogemm.gemm(H(q), H(s), H(wt), H(wts)))
                  <= 1e-5 * ogemm.abs_bound(H(q), H(s), H(wt), H(wts)))
    assert np.all(np.abs(_value(dw) - ogemm.gemm_rowscaled(H(qt), H(st), H(xt), H(xts)))
                  <= 1e-5 * ogemm.abs_bound_rowscaled(H(qt), H(st), H(xt), H(xts)))
    # and the whole step against unquantized gradients: E4M3 keeps 2^-4, and
    # errors of that size add up like a random walk over the products
    Y = _value(x) @ _value(w).T
    dY = off.gated_backward("silu", _value(dh), Y)
    for got, ref in ((_value(dx), dY @ _value(w)), (_value(dw), dY.T @ _value(x))):
        assert np.linalg.norm(got - ref) <= 0.1 * np.linalg.norm(ref)


def test_example_trains_and_serves(capsys):
    """examples/feed_forward.py at a small size: the loss falls, INT8 serving
    stays near the FP8 layer, the grouped call near each expert's own."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward_example", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses = ex.main(["--tokens", "512", "--hidden", "256", "--ffn", "256", "--steps", "12",
                      "--lr", "100"])
    assert losses[-1] < 0.9 * losses[0]
    out = capsys.readouterr().out
    assert float(out.split("served in INT8: ")[1].split()[0]) < 0.1
    assert float(out.split("within ")[1].split()[0]) < 1e-2
