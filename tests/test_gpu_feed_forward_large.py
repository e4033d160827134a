"""The feed-forward calls at sizes that take each tile size, and past 32-bit
offsets.

The block-scaled tiles add an output's chunks in the same order as fp8q_gemm,
so the saved pre-activations must be its BF16 rounding bit for bit (fp8q_gemm
itself is held to its bound elsewhere).  int8 sums are exact: the reference is a
float64 product on the GPU.  Tolerances as in test_gpu_feed_forward.
"""

import numpy as np
import pytest
import torch

from gpu_util import DEV, fq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i8(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int8)


def _pos(g, *shape):
    return torch.rand(shape, generator=g, device=DEV) * 1e-2 + 1e-3


def _bits(t):
    return t.view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()])


def _act(act, x):
    y = x if act == "silu" else 2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
    return x * torch.sigmoid(y), y


def _close(got, ref, rel):
    """|got - ref| <= rel |ref|, and half a BF16 ulp (2^-8 relative, with the
    same slack as elsewhere) for BF16 output."""
    half = 2.0 ** -8 * (1 + 2.0 ** -6) if got.dtype == torch.bfloat16 else 0.0
    return bool(((got.double() - ref).abs() <= (rel + half) * ref.abs() + 1e-36).all())


# 64-, 128- and 256-row tiles; N odd, K with a part of a chunk
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,bias", [(600, 1030, 336, True), (1633, 6456, 336, False),
                                        (3000, 4099, 656, True), (2050, 4100, 208, False),
                                        (4097, 8192, 1040, False)])
def test_gemm_i8_tiles(M, N, K, bias, out):
    g = _gen(M + N)
    a, w, sa, sw = _i8(g, M, K), _i8(g, N, K), _pos(g, M), _pos(g, N)
    b = torch.randn(N, generator=g, device=DEV) if bias else None
    c = fq().gemm_i8(a, sa, w, sw, bias=b, out_dtype=out)
    p = (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double()
    if b is None:
        assert _close(c, p, 4 * U)
    else:
        ref = p + b.double()
        half = 2.0 ** -8 * (1 + 2.0 ** -6) if out == torch.bfloat16 else 0.0
        tol = 4 * U * (p.abs() + b.double().abs()) + half * ref.abs()
        assert bool(((c.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", [(700, 261, 336), (1000, 2000, 336), (3000, 2050, 1040),
                                   (4097, 4096, 784)])
def test_gemm_i8_gated_tiles(M, F, K, act):
    g = _gen(M + F)
    a, w, sa, sw = _i8(g, M, K), _i8(g, 2 * F, K), _pos(g, M), _pos(g, 2 * F)
    sw = sw * (2.0 / (5400 * K ** 0.5 * 6e-3 * 6e-3))      # gates of order 2
    p = (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double()
    x, y = _act(act, p[:, :F])
    ref = x * p[:, F:]
    # both factors carry 4u; the gate's is multiplied by its condition 1 + |y|
    rel = U * (16 + 8 * y.abs() + 4 * (1 + 3 * y.abs()) + 8)
    for out in (torch.bfloat16, torch.float32):
        assert _close(fq().gemm_i8_gated(a, sa, w, sw, act=act, out_dtype=out), ref, rel)


# the tiles of 32 and 64 rows: one row in the last tile, one column, one chunk of
# K and part of it, chunks that end inside the ring's first round
@pytest.mark.parametrize("M,N,K,bias", [(33, 70, 16, True), (65, 300, 1040, False),
                                        (333, 1100, 1040, True), (500, 2051, 336, False),
                                        (449, 2001, 400, True), (129, 513, 2064, False),
                                        (17, 16390, 256, True), (32, 16384, 144, False)])
def test_gemm_i8_small_tiles(M, N, K, bias):
    for out in (torch.bfloat16, torch.float32):
        test_gemm_i8_tiles(M, N, K, bias, out)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", [(33, 35, 144), (97, 150, 1040), (450, 1000, 336),
                                   (513, 1025, 528), (20, 8200, 256)])
def test_gemm_i8_gated_small_tiles(M, F, K, act):
    test_gemm_i8_gated_tiles(M, F, K, act)


# 256 x 128 tiles
@pytest.mark.parametrize("M,N,K,bias", [(1793, 4001, 1808, True), (2048, 4096, 2064, False)])
def test_gemm_i8_middle_tiles(M, N, K, bias):
    for out in (torch.bfloat16, torch.float32):
        test_gemm_i8_tiles(M, N, K, bias, out)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gemm_i8_gated_middle_tiles(act):
    test_gemm_i8_gated_tiles(1793, 2005, 1808, act)


def _codes(g, *shape):
    """E4M3 codes of finite values."""
    return torch.randint(0, 127, shape, generator=g, device=DEV, dtype=torch.uint8) \
        + 128 * torch.randint(0, 2, shape, generator=g, device=DEV, dtype=torch.uint8)


def _gated_inputs(g, M, F, K, G=None):
    lead = () if G is None else (G,)
    # code values have a root mean square of about 130: sums of order 2
    sa = _pos(g, K // 128, M) * (2.0 / (130 ** 2 * K ** 0.5 * 6e-3 * 6e-3))
    return (_codes(g, M, K), sa, _codes(g, *lead, 2 * F, K),
            _pos(g, *lead, 2 * F // 128, K // 128))


def _check_h(h, y, F, act):
    """h against act of the FP32 pre-activations that both paths form alike."""
    x, arg = _act(act, y[:, :F].double())
    assert _close(h, x * y[:, F:].double(), U * (24 + 8 * arg.abs()))


@pytest.mark.parametrize("M,F,K,act", [(520, 640, 128, "silu"), (2000, 1024, 256, "gelu_tanh"),
                                       (7600, 896, 128, "silu"), (4097, 2048, 512, "silu"),
                                       (8190, 2176, 896, "gelu_tanh")])
def test_gemm_gated_tiles_form_the_gemms_sums(M, F, K, act):
    f, g = fq(), _gen(M + F)
    a, sa, w, sw = _gated_inputs(g, M, F, K)
    y = f.gemm(a, sa, w, sw)
    for out in (torch.bfloat16, torch.float32):
        h, gu = f.gemm_gated(a, sa, w, sw, act=act, out_dtype=out, save_gate_up=True)
        assert torch.equal(_bits(gu), _bits(y.to(torch.bfloat16)))
        _check_h(h, y, F, act)
        assert torch.equal(_bits(f.gemm_gated(a, sa, w, sw, act=act, out_dtype=out)), _bits(h))


# 128 x 128 and 256 x 128 tiles, one row in the last of them
@pytest.mark.parametrize("M,F,K,act", [(641, 2048, 512, "gelu_tanh"), (900, 2048, 256, "silu"),
                                       (1537, 1664, 512, "gelu_tanh"), (2048, 2048, 1664, "silu")])
def test_gemm_gated_middle_tiles_form_the_gemms_sums(M, F, K, act):
    test_gemm_gated_tiles_form_the_gemms_sums(M, F, K, act)


def test_grouped_gemm_gated_forms_the_grouped_gemms_sums():
    """Every row-count bucket of the grouped kernel, empty experts among them."""
    f, g = fq(), _gen(7)
    counts = [0, 1, 63, 64, 65, 128, 129, 160, 161, 192, 193, 256, 257, 300, 0, 520, 17, 0]
    F, K = 384, 640
    ends = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
    M = int(ends[-1]) + 5
    a, sa, w, sw = _gated_inputs(g, M, F, K, len(counts))
    n = int(ends[-1])
    y = f.grouped_gemm(a, sa, ends, w, sw)[:n]
    h, gu = f.grouped_gemm_gated(a, sa, ends, w, sw, save_gate_up=True)
    assert torch.equal(_bits(gu[:n]), _bits(y.to(torch.bfloat16)))
    _check_h(h[:n], y, F, "silu")


# ------------------------------------------------------------- past 32-bit offsets
@pytest.mark.parametrize("M", [2, 100])
def test_gemm_i8_weights_past_4_gib(M):
    g, N, K = _gen(M), 40000, 131056
    a, w, sa, sw = _i8(g, M, K), _i8(g, N, K), _pos(g, M), _pos(g, N)
    c = fq().gemm_i8(a, sa, w, sw)
    at = torch.tensor([0, 1, 16383, 16384, 16385, 32767, 32768, 32769, N - 130, N - 1], device=DEV)
    ref = (a.double() @ w[at].double().t()) * sa.double()[:, None] * sw[at].double()
    assert _close(c[:, at], ref, 4 * U)
    sa = sa * (2.0 / (5400 * K ** 0.5 * 6e-3 * 6e-3))      # gates of order 2
    h = fq().gemm_i8_gated(a, sa, w, sw, out_dtype=torch.float32)
    up = at[:5]
    p = [(a.double() @ w[r].double().t()) * sa.double()[:, None] * sw[r].double()
         for r in (up, N // 2 + up)]
    x, y = _act("silu", p[0])
    assert _close(h[:, up], x * p[1], U * (40 + 24 * y.abs()))


def test_gemm_i8_output_past_2_31_elements():
    g, M, N, K = _gen(3), 70001, 40000, 64
    a, w, sa, sw = _i8(g, M, K), _i8(g, N, K), _pos(g, M), _pos(g, N)
    c = fq().gemm_i8(a, sa, w, sw, out_dtype=torch.bfloat16)
    at = torch.tensor([0, 53686, 53687, 53688, 60000, M - 129, M - 1], device=DEV)
    ref = (a[at].double() @ w.double().t()) * sa[at].double()[:, None] * sw.double()
    assert _close(c[at], ref, 4 * U)


def test_gemm_gated_weights_past_4_gib():
    f, g, F, K = fq(), _gen(5), 40960, 57344
    for M in (3, 129):
        a, sa, w, sw = _gated_inputs(g, M, F, K)
        h = f.gemm_gated(a, sa, w, sw)
        for f0 in (0, 36864, F - 128):      # a block of features alone: the same sums
            r = torch.cat([torch.arange(f0, f0 + 128), F + torch.arange(f0, f0 + 128)]).to(DEV)
            b = torch.tensor([f0 // 128, (F + f0) // 128], device=DEV)
            y = f.gemm(a, sa, w[r].contiguous(), sw[b].contiguous(), precise=True)
            x, arg = _act("silu", y[:, :128].double())
            ref = x * y[:, 128:].double()
            # the FP8 product against the precise one: norms, not element by element
            got = h[:, f0:f0 + 128].double()
            assert (got - ref).norm() <= 5e-3 * ref.norm()


def test_gated_backward_past_2_31_elements():
    """Any 128 tokens of a large batch are the same 128 tokens alone."""
    f, g, M, F = fq(), _gen(9), 270000, 4096
    dh = (torch.randn((M, F), generator=g, device=DEV, dtype=torch.bfloat16)) * 0.01
    gu = torch.randn((M, 2 * F), generator=g, device=DEV, dtype=torch.bfloat16)
    q, s, qt, st = f.gated_backward(dh, gu)
    for t0 in (0, 128 * 1023, 128 * 2047, 128 * 2048, M // 128 * 128):
        t1 = min(M, t0 + 128)
        q1, s1, qt1, st1 = f.gated_backward(dh[t0:t1], gu[t0:t1])
        assert torch.equal(q[t0:t1], q1) and torch.equal(s[:, t0:t1], s1)
        assert torch.equal(qt[:, t0:t0 + 128], qt1) and torch.equal(st[t0 // 128], st1[0])


def test_quantize_token_i8_past_2_31_elements():
    f, g, M, K = fq(), _gen(10), 300001, 8191
    x = torch.randn((M, K), generator=g, device=DEV, dtype=torch.bfloat16)
    q, s = f.quantize_token_i8(x)
    for r in (0, 262175, 262176, 262177, M - 1):
        q1, s1 = f.quantize_token_i8(x[r:r + 1].clone())
        assert torch.equal(q[r:r + 1], q1) and torch.equal(s[r:r + 1], s1)
