"""Tokens grouped by expert: the quantizer along the tokens, the gated block's
backward pass and the weight gradients, on the GPU.

The codes are bit for bit those of the dense calls on each expert's rows, padded
with zeros to whole groups; the products hold the bounds of the dense row-scaled
calls, expert by expert (gpu_util.assert_gemm_bounded, assert_gemm_strict)."""

import ctypes

import numpy as np
import pytest
import torch

import workloads
from gpu_util import DEV, assert_gemm_bounded, assert_gemm_strict, bf16_to_bits, fq, host, to_dev_bf16
from oracle import quant as oquant, training_step as ots
from test_gpu_offsets import E_OFFSETS, LIB_DEBUG, OK

pytestmark = pytest.mark.gpu

# rows of each expert, and rows past the last
SPLITS = {
    "one expert": ([200], 0),
    "one row": ([1], 0),
    "none": ([0, 0, 0], 0),
    "none, rows behind": ([0, 0], 70),
    "whole groups": ([128, 256, 128], 0),
    "ragged": ([0, 1, 127, 128, 129, 0, 300, 5], 0),
    "rows behind": ([64, 0, 130], 200),
    "first and last empty": ([0, 250, 0], 3),
    "many experts, few rows": ([(3 * e) % 4 for e in range(70)], 0),
    "1024 experts": ([1 if e % 5 == 0 else 0 for e in range(1024)], 0),
    "65 experts": ([e % 7 * 40 for e in range(65)], 9),
}


def _split(name):
    n, behind = SPLITS[name]
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    return off, int(off[-1]) + behind, torch.from_numpy(off).to(DEV)


def _bits(rng, M, K, scale=1.0):
    return workloads.bf16_bits((scale * rng.standard_normal((M, K))
                                * np.exp(rng.uniform(-2, 2, (M, 1)))).astype(np.float32))


@pytest.mark.parametrize("mode", ["f32", "pow2"])
@pytest.mark.parametrize("name", list(SPLITS))
def test_grouped_quantize_act_t(name, mode):
    off, M, off_d = _split(name)
    rng = np.random.default_rng([len(off), M])
    for K in (128, 384):
        x = _bits(rng, M, K)
        q, s = fq().grouped_quantize_act_t(to_dev_bf16(x), off_d, mode)
        T = fq().expert_columns(M, len(off) - 1)
        assert q.shape == (K, T) and s.shape == (T // 128, K)
        rq, rs = oquant.quantize_act_t(ots.expert_rows(x, off, T), mode)
        assert np.array_equal(host(q), rq)
        assert np.array_equal(host(s).view(np.uint32), rs.view(np.uint32))


@pytest.mark.parametrize("act,mode", [("silu", "f32"), ("gelu_tanh", "f32"), ("silu", "pow2")])
@pytest.mark.parametrize("name,F", [(n, 128) for n in SPLITS] +
                         [("ragged", 512), ("ragged", 2048), ("65 experts", 256),
                          ("rows behind", 4096)])
def test_grouped_gated_backward(name, F, act, mode):
    """Both kernels of the dense call (small pieces and whole blocks), by expert."""
    off, M, off_d = _split(name)
    rng = np.random.default_rng([F, M])
    dh, gu = to_dev_bf16(_bits(rng, M, F, 0.1)), to_dev_bf16(_bits(rng, M, 2 * F))
    f, T = fq(), fq().expert_columns(M, len(off) - 1)
    q = torch.full((M, 2 * F), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((2 * F // 128, M), -3.0, device=DEV)
    qt = torch.full((2 * F, T), 0x55, dtype=torch.uint8, device=DEV)
    st = torch.full((T // 128, 2 * F), -3.0, device=DEV)
    f.fp8q_grouped_gated_backward(dh, gu, off_d, q, s, qt, st, act, mode)
    end = int(off[-1])
    want_qt, want_st = torch.zeros_like(qt), torch.zeros_like(st)
    if end:
        rq, rs, _, _ = f.gated_backward(dh[:end], gu[:end], act, mode)
        assert torch.equal(q[:end], rq) and torch.equal(s[:, :end], rs)
    assert (q[end:] == 0x55).all() and (s[:, end:] == -3.0).all()
    at = 0
    for lo, hi in zip(off[:-1], off[1:]):
        if hi > lo:
            _, _, rqt, rst = f.gated_backward(dh[lo:hi], gu[lo:hi], act, mode)
            want_qt[:, at:at + rqt.shape[1]] = rqt
            want_st[at // 128:at // 128 + rst.shape[0]] = rst
            at += rqt.shape[1]
    # (a code of a zero can have either sign; those of padding are +0)
    assert torch.equal(qt, want_qt) and torch.equal(st, want_st)
    # one pair alone gives the same
    r = f.grouped_gated_backward(dh, gu, off_d, act, mode, rows=False)
    assert r[0] is None and torch.equal(r[2], qt) and torch.equal(r[3], st)
    r = f.grouped_gated_backward(dh, gu, off_d, act, mode, tokens=False)
    assert r[2] is None and torch.equal(r[0][:end], q[:end]) and torch.equal(r[1][:, :end], s[:, :end])


def _operands(off, M, off_d, N, K, seed, outliers=False):
    rng = np.random.default_rng([seed, N, K])
    a, b = _bits(rng, M, N, 0.02), _bits(rng, M, K)
    if outliers:
        b = workloads.bf16_bits(oquant.bf16_bits_to_f32(b) * np.where(rng.random(K) < 0.05, 50, 1)
                                .astype(np.float32))
    return (*fq().grouped_quantize_act_t(to_dev_bf16(a), off_d),
            *fq().grouped_quantize_act_t(to_dev_bf16(b), off_d))


def _check(c, operands, off, out, precise, what):
    qa, sa, qb, sb = [host(t) for t in operands]
    at = 0
    for e in range(len(off) - 1):
        w = -(-(off[e + 1] - off[e]) // 128) * 128
        if w == 0:
            assert not c[e].any(), f"{what}: expert {e} has no tokens"
            continue
        cols, g = slice(at, at + w), slice(at // 128, (at + w) // 128)
        at += w
        got = oquant.bf16_bits_to_f32(bf16_to_bits(c[e])) if out == "bf16" else host(c[e])
        check = assert_gemm_strict if precise else assert_gemm_bounded
        check(got, np.ascontiguousarray(qa[:, cols]), sa[g], np.ascontiguousarray(qb[:, cols]),
              sb[g], out, f"{what}, expert {e}", rowscaled=True)


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("name,N,K", [(n, 128, 128) for n in SPLITS if n != "1024 experts"] +
                         [("1024 experts", 128, 128), ("ragged", 384, 256), ("ragged", 128, 640),
                          ("rows behind", 256, 1024), ("one expert", 512, 384),
                          ("whole groups", 640, 128)])
def test_grouped_gemm_rowscaled(name, N, K, out, precise):
    off, M, off_d = _split(name)
    ops = _operands(off, M, off_d, N, K, 1, outliers=N == K)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    c = fq().grouped_gemm_rowscaled(*ops, off_d, out_dtype=dt, precise=precise)
    assert c.shape == (len(off) - 1, N, K) and c.dtype == dt
    _check(c, ops, off, out, precise, f"{name} {N}x{K}")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("name,N,K", [("65 experts", 640, 1664), ("65 experts", 640, 1152),
                                      ("1024 experts", 128, 384), ("ragged", 4224, 7296),
                                      ("rows behind", 1024, 128), ("first and last empty", 128, 1024)])
def test_every_tile_size_equals_the_dense_call(name, N, K, out):
    """Large and small tiles, ending inside the outputs in both directions: each
    expert's gradient is the dense call's on its columns, bit for bit (the same sums
    in the same order)."""
    off, M, off_d = _split(name)
    qa, sa, qb, sb = _operands(off, M, off_d, N, K, 7)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    c = fq().grouped_gemm_rowscaled(qa, sa, qb, sb, off_d, out_dtype=dt)
    at = 0
    for e in range(len(off) - 1):
        w = -(-int(off[e + 1] - off[e]) // 128) * 128
        if w == 0:
            assert not c[e].any()
            continue
        cols, g = slice(at, at + w), slice(at // 128, (at + w) // 128)
        at += w
        want = fq().gemm_rowscaled(qa[:, cols].contiguous(), sa[g], qb[:, cols].contiguous(), sb[g],
                                   out_dtype=dt)
        assert torch.equal(c[e], want), f"expert {e}"


@pytest.mark.parametrize("tokens", [1000, 2500])
def test_grouped_gemm_rowscaled_long(tokens):
    """Experts of many groups, and one expert's gradient against the dense call's."""
    n = [tokens, 17, 2 * tokens, 384]
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    off_d = torch.from_numpy(off).to(DEV)
    ops = _operands(off, int(off[-1]), off_d, 256, 384, 3)
    for precise in (False, True):
        c = fq().grouped_gemm_rowscaled(*ops, off_d, precise=precise)
        _check(c, ops, off, "f32", precise, "long")


def test_more_columns_than_asked_for():
    """T past the experts' groups is not read, however large."""
    off, M, off_d = _split("ragged")
    qa, sa, qb, sb = _operands(off, M, off_d, 128, 256, 5)
    want = fq().grouped_gemm_rowscaled(qa, sa, qb, sb, off_d)

    def wider(q, s):
        q2 = torch.full((q.shape[0], q.shape[1] + 1024), 0x7F, dtype=torch.uint8, device=DEV)
        s2 = torch.full((s.shape[0] + 8, s.shape[1]), float("nan"), device=DEV)
        q2[:, :q.shape[1]], s2[:s.shape[0]] = q, s
        return q2, s2
    assert torch.equal(fq().grouped_gemm_rowscaled(*wider(qa, sa), *wider(qb, sb), off_d), want)


def test_columns_past_32_bit_offsets():
    """A tile's rows of 2^24 columns: the last bytes of the operands are past 2^31 of
    a tile's first, and past 2^32 of the operand's."""
    T, N, K = 1 << 24, 256, 128
    lead = T - 512
    off_d = torch.tensor([0, 0, T], dtype=torch.int32, device=DEV)
    qa = torch.zeros((N, T), dtype=torch.uint8, device=DEV)
    qb = torch.zeros((K, T), dtype=torch.uint8, device=DEV)
    sa = torch.zeros((T // 128, N), device=DEV)
    sb = torch.zeros((T // 128, K), device=DEV)
    rng = np.random.default_rng(6)
    ops = []
    for q, s, w in ((qa, sa, N), (qb, sb, K)):
        tq, ts = fq().quantize_act_t(to_dev_bf16(_bits(rng, 512, w)))
        q[:, lead:], s[lead // 128:] = tq, ts
        ops += [tq, ts]
    c = fq().grouped_gemm_rowscaled(qa, sa, qb, sb, off_d)
    want = fq().gemm_rowscaled(*ops)
    assert not c[0].any()
    # the sums begin with exact zeros, so the last four groups' come out the same
    assert torch.equal(c[1], want)


# ----------------------------------------------------------------- invalid offsets
BAD = {"first not zero": [1, 10, 20, 30], "decreasing": [0, 50, 40, 60],
       "past the end": [0, 10, 20, 101], "negative": [0, -5, 20, 30]}
ROWS, K3, F3 = 512, 128, 128


def _calls(L, off):
    """{call: (status, its outputs)}: outputs are filled before."""
    d_off = torch.tensor(off, dtype=torch.int32, device=DEV)
    G, st = len(off) - 1, torch.cuda.current_stream().cuda_stream
    M, T = 100, 128 * (512 // 128 + G)
    x = torch.ones((ROWS, K3), dtype=torch.bfloat16, device=DEV)
    gu = torch.ones((ROWS, 2 * F3), dtype=torch.bfloat16, device=DEV)
    fill8 = lambda *s: torch.full(s, 0x55, dtype=torch.uint8, device=DEV)   # noqa: E731
    fill = lambda *s: torch.full(s, -3.0, device=DEV)   # noqa: E731
    out = {}
    q, s = fill8(K3, T), fill(T // 128, K3)
    r = L.fp8q_grouped_quantize_act_t(x.data_ptr(), M, d_off.data_ptr(), G, K3, q.data_ptr(),
                                      s.data_ptr(), 0, st)
    out["quantize"] = r, [q, s]
    o = [fill8(ROWS, 2 * F3), fill(2, ROWS), fill8(2 * F3, T), fill(T // 128, 2 * F3)]
    r = L.fp8q_grouped_gated_backward(x.data_ptr(), gu.data_ptr(), M, d_off.data_ptr(), G, F3, 0, 0,
                                      *[t.data_ptr() for t in o], st)
    out["backward"] = r, o
    a, sa = torch.ones((128, T), dtype=torch.uint8, device=DEV), torch.ones((T // 128, 128), device=DEV)
    for name in ("fp8q_grouped_gemm_rowscaled", "fp8q_grouped_gemm_rowscaled_precise"):
        c = fill(G, 128, 128)
        r = getattr(L, name)(a.data_ptr(), sa.data_ptr(), a.data_ptr(), sa.data_ptr(), 256,
                             d_off.data_ptr(), G, 128, 128, c.data_ptr(), 0, st)
        out[name] = r, [c]
    torch.cuda.synchronize()
    return out


def _debug():
    L = ctypes.CDLL(LIB_DEBUG)
    for n in ("fp8q_grouped_quantize_act_t", "fp8q_grouped_gated_backward",
              "fp8q_grouped_gemm_rowscaled", "fp8q_grouped_gemm_rowscaled_precise"):
        getattr(L, n).argtypes = getattr(fq().lib, n).argtypes
        getattr(L, n).restype = getattr(fq().lib, n).restype
    return L


def _untouched(outs):
    return all(bool((t == (0x55 if t.dtype == torch.uint8 else -3.0)).all()) for t in outs)


@pytest.mark.parametrize("case", list(BAD))
def test_release_build_writes_nothing_for_invalid_offsets(case):
    # (the gradient knows no number of rows: there 101 rows are too many groups)
    for name, (r, outs) in _calls(fq().lib, BAD[case]).items():
        gemm = name.startswith("fp8q")
        if gemm and case == "past the end":
            continue
        assert r == OK and _untouched(outs), name
    off = [0, 100, 300, 500]      # more groups than the operands' 256 columns hold
    for name, (r, outs) in _calls(fq().lib, off).items():
        assert r == OK and _untouched(outs), name


def test_debug_build_reports_invalid_offsets():
    L = _debug()
    for case, bad in BAD.items():
        for name, (r, outs) in _calls(L, bad).items():
            if name.startswith("fp8q") and case == "past the end":
                continue
            assert r == E_OFFSETS and _untouched(outs), (case, name)
        good = [0, 40, 40, 100]   # and the flag has been cleared
        for (name, (r, outs)), (r2, outs2) in zip(_calls(L, good).items(),
                                                  _calls(fq().lib, good).values()):
            assert r == r2 == OK, name
            for a, b in zip(outs, outs2):
                assert torch.equal(a, b), name


@pytest.mark.parametrize("mode", ["f32", "pow2"])
def test_grouped_gated_backward_of_many_groups_is_each_experts_own(mode):
    """Enough groups that a workgroup takes several blocks of features, the last one fewer:
    every expert's codes are those of a call for it alone, bit for bit."""
    G, F, M = 200, 17 * 128, 20000
    rng = np.random.default_rng(12)
    counts = rng.integers(0, 150, size=G)
    counts[[0, 7, 199]] = 0, 700, 0
    off = np.concatenate([[0], np.cumsum(counts)])
    assert off[-1] < M
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    dh = torch.randn((M, F), generator=g, device=DEV).to(torch.bfloat16)
    gu = torch.randn((M, 2 * F), generator=g, device=DEV).to(torch.bfloat16)
    offd = torch.from_numpy(off.astype(np.int32)).to(DEV)
    q, s, qt, st = fq().grouped_gated_backward(dh, gu, offd, mode=mode)
    at = 0
    for e in range(G):
        lo, hi = int(off[e]), int(off[e + 1])
        n = -(-(hi - lo) // 128)
        if n:
            eq, es, eqt, est = fq().gated_backward(dh[lo:hi].clone(), gu[lo:hi].clone(), mode=mode)
            assert torch.equal(q[lo:hi], eq) and torch.equal(s[:, lo:hi], es), e
            assert torch.equal(qt[:, 128 * at:128 * (at + n)], eqt), e
            assert torch.equal(st[at:at + n], est), e
        at += n
    assert not qt[:, 128 * at:].any() and not st[at:].any()
