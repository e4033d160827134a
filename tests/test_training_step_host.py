"""Layer norm, tokens by expert and AdamW without a GPU: the oracle against
differences, its dither, the column bound, host-side refusals of the C ABI and of
the binding."""

import ctypes
import os
import unittest.mock as um

import numpy as np
import pytest
import torch

from oracle import e4m3, training_step as ots

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
fq = pytest.importorskip("fine_grained_block_fp8q_amd")

OK, E_NULL, E_SHAPE, E_ALIGN, E_ENUM, E_DEVICE, E_LAUNCH, E_UNSUP, E_OFFSETS = range(9)
u8, f32, bf16, i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32
A = 0x10000  # a fake aligned address: never dereferenced on these paths
NAMES = ["fp8q_layer_norm", "fp8q_layer_norm_backward", "fp8q_layer_norm_backward_workspace",
         "fp8q_expert_columns", "fp8q_grouped_quantize_act_t", "fp8q_grouped_gated_backward",
         "fp8q_grouped_gemm_rowscaled", "fp8q_grouped_gemm_rowscaled_precise", "fp8q_adamw"]


# ------------------------------------------------------------------- the oracle
def test_oracle_layer_norm_gradient_against_differences():
    """Central differences of step 1e-5 of sum(dy y): off by h^2/6 of the third
    derivative (of order 10 here) and eps/h of values of order 10, under 1e-7."""
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 9)), rng.standard_normal((3, 9))
    w, b, eps, h = rng.standard_normal(9), rng.standard_normal(9), 1e-3, 1e-5
    _, mean, rstd = ots.layer_norm(x, w, b, eps)
    dx, dw, db = ots.layer_norm_backward(dy, x, w, mean, rstd)
    f = lambda x, w, b: (dy * ots.layer_norm(x, w, b, eps)[0]).sum()   # noqa: E731
    for grad, at in ((dx, 0), (dw, 1), (db, 2)):
        for i in np.ndindex(grad.shape):
            p, m = [[t.copy() for t in (x, w, b)] for _ in range(2)]
            p[at][i] += h
            m[at][i] -= h
            assert abs((f(*p) - f(*m)) / (2 * h) - grad[i]) < 1e-7


def test_oracle_moments_are_the_recurrence():
    """At t = 1 from zero moments the corrected moments are g and g^2: p moves by
    lr sign(g) g/(|g| + eps)."""
    g = np.array([0.5, -2.0, 1e-3, 0.0], dtype=np.float32)
    m, v = ots.adamw_moments(np.zeros(4), np.zeros(4), g, 0.9, 0.95)
    p, up = ots.adamw_parameters(np.ones(4), m, v, 1, 0.1, 0.9, 0.95, 1e-8, 0.0)
    assert np.allclose(up, 0.1 * np.sign(g), rtol=3e-5) and np.allclose(p, 1 - up)


def test_dither_keeps_the_mean():
    """Codes of one value over 1000 steps average to it: u of one element is spread
    so evenly over the steps (a sequence of the golden ratio) that the share of
    steps rounded up is off its value by less than (ln 1000)/1000 + 2^-20."""
    for x in (1.03, 3.9, 100.7, 0.0131, 0.0007):
        v = np.zeros(128, dtype=np.float32)
        v[0], v[1:] = 448.0, x
        r = np.mean([e4m3.decode(ots.encode_moments(v, t)[0]) for t in range(1, 1001)], axis=0)
        step = 2.0 ** (max(np.floor(np.log2(x)), -6) - 3)
        assert np.abs(r[1:] - np.float32(x)).max() < 0.01 * step


def test_encoded_moments_stay_within_a_step():
    """Each code stands for a value within one step of E4M3 of the given one."""
    rng = np.random.default_rng(5)
    x = (rng.standard_normal(1000) * np.exp(rng.uniform(-9, 3, 1000))).astype(np.float32)
    q, s = ots.encode_moments(x, 7)
    wide = np.repeat(s.astype(np.float64), 128)[:1000]
    y = np.abs(x) / wide
    step = 2.0 ** (np.maximum(np.floor(np.log2(y)), -6) - 3)
    assert np.all(np.abs(ots.decode_moments(q, s) - x) <= wide * step * (1 + 1e-5))
    assert np.all(np.sign(ots.decode_moments(q, s)) * np.sign(x) >= 0)
    root = np.abs(x) * 1e-6
    root[::128] = 1.0
    q, s = ots.encode_moments(root, 9, second=True)
    assert np.all(ots.decode_moments(q, s) > 0)


def test_expert_columns_bound():
    """Enough for any split of M rows over G experts, and the least that is."""
    rng = np.random.default_rng(2)
    for G in (1, 2, 3, 7, 40, 1024):
        for M in (0, 1, 2, 3, 127, 128, 129, 500, 4096, 100000):
            T = fq.expert_columns(M, G)
            assert T % 128 == 0
            worst = 0
            for _ in range(20):
                cut = np.sort(rng.integers(0, M + 1, G - 1))
                n = np.diff(np.concatenate([[0], cut, [M]]))
                worst = max(worst, int((-(-n // 128)).sum()) * 128)
            assert worst <= T
            # one token to each of all but one expert, and the rest where it
            # leaves the most groups unfilled
            e = min(G, M)
            if e:
                full = (M - e) // 128          # groups beyond the first of each
                assert T == 128 * (e + full)
    assert fq.expert_columns(0, 5) == 0


# -------------------------------------------------------------------- the C ABI
@pytest.fixture(params=["libfp8q.so", "libfp8q_debug.so"])
def lib(request):
    L = ctypes.CDLL(os.path.join(ROOT, "fine_grained_block_fp8q_amd", request.param))
    for n in NAMES:
        getattr(L, n).argtypes = getattr(fq.lib, n).argtypes
        getattr(L, n).restype = getattr(fq.lib, n).restype
    return L


def test_layer_norm_refusals(lib):
    f = lib.fp8q_layer_norm
    good = [A, 1, A, A, 4, 256, 1e-5, A, 1, A, A, 0, A, A, None]

    def call(**at):
        a = list(good)
        for k, v in at.items():
            a[int(k[1:])] = v
        return f(*a)
    for i in (0, 2, 12, 13):
        assert call(**{f"_{i}": None}) == E_NULL
    assert call(_9=None) == E_NULL and call(_10=None) == E_NULL
    assert call(_7=None, _9=None, _10=None) == E_NULL
    assert call(_4=-1) == E_SHAPE and call(_5=0) == E_SHAPE and call(_5=200) == E_SHAPE
    for i in (0, 7, 9):
        assert call(**{f"_{i}": A + 8}) == E_ALIGN
    for i in (2, 3, 10, 12, 13):
        assert call(**{f"_{i}": A + 2}) == E_ALIGN
    assert call(_1=2) == E_ENUM and call(_8=2) == E_ENUM and call(_11=2) == E_ENUM
    assert call(_5=16384 + 128) == E_UNSUP
    for eps in (-1e-5, float("nan"), float("inf")):
        assert call(_6=eps) == E_UNSUP
    assert f(None, 1, None, None, 0, 256, 0.0, None, 1, None, None, 0, None, None, None) == OK


def test_layer_norm_backward_refusals(lib):
    f = lib.fp8q_layer_norm_backward
    good = [A, 1, A, 1, A, A, A, 40, 200, A, A, A, A, None]

    def call(**at):
        a = list(good)
        for k, v in at.items():
            a[int(k[1:])] = v
        return f(*a)
    for i in (0, 2, 4, 5, 6, 9, 10, 12):
        assert call(**{f"_{i}": None}) == E_NULL
    assert call(_7=-1) == E_SHAPE and call(_8=0) == E_SHAPE
    for i in (0, 2, 9, 12):
        assert call(**{f"_{i}": A + 8}) == E_ALIGN
    for i in (4, 5, 6, 10, 11):
        assert call(**{f"_{i}": A + 2}) == E_ALIGN
    assert call(_1=2) == E_ENUM and call(_3=2) == E_ENUM
    assert call(_8=16385) == E_UNSUP
    w = lib.fp8q_layer_norm_backward_workspace
    assert w(0, 100) == 0 and w(5, 0) == 0 and w(-1, 100) == 0 and w(5, 16385) == 0
    assert w(1, 100) == 0          # one workgroup writes the results itself
    assert w(100, 100) > 0 and w(1 << 40, 16384) >= w(4096, 16384) > 0


def test_grouped_refusals(lib):
    f = lib.fp8q_grouped_quantize_act_t
    assert f(None, 8, A, 2, 128, A, A, 0, None) == E_NULL
    assert f(A, 8, None, 2, 128, A, A, 0, None) == E_NULL
    assert f(A, 8, A, 2, 128, None, A, 0, None) == E_NULL
    assert f(A, 8, A, 2, 128, A, None, 0, None) == E_NULL
    assert f(A, -8, A, 2, 128, A, A, 0, None) == E_SHAPE
    assert f(A, 1 << 31, A, 2, 128, A, A, 0, None) == E_SHAPE
    assert f(A, 8, A, 0, 128, A, A, 0, None) == E_SHAPE
    assert f(A, 8, A, 2, 64, A, A, 0, None) == E_SHAPE
    assert f(A + 8, 8, A, 2, 128, A, A, 0, None) == E_ALIGN
    assert f(A, 8, A + 2, 2, 128, A, A, 0, None) == E_ALIGN
    assert f(A, 8, A, 2, 128, A + 8, A, 0, None) == E_ALIGN
    assert f(A, 8, A, 2, 128, A, A + 2, 0, None) == E_ALIGN
    assert f(A, 8, A, 2, 128, A, A, 2, None) == E_ENUM
    assert f(A, 8, A, 1025, 128, A, A, 0, None) == E_UNSUP
    assert f(A, 8, A, 2, (1 << 22) + 128, A, A, 0, None) == E_UNSUP
    assert f(None, 0, A, 2, 128, None, None, 0, None) == OK

    f = lib.fp8q_grouped_gated_backward
    assert f(None, A, 8, A, 2, 128, 0, 0, A, A, A, A, None) == E_NULL
    assert f(A, A, 8, None, 2, 128, 0, 0, A, A, A, A, None) == E_NULL
    assert f(A, A, 8, A, 2, 128, 0, 0, A, None, A, A, None) == E_NULL
    assert f(A, A, 8, A, 2, 128, 0, 0, None, None, None, None, None) == E_NULL
    assert f(A, A, 8, A, 0, 128, 0, 0, A, A, A, A, None) == E_SHAPE
    assert f(A, A, 8, A, 2, 100, 0, 0, A, A, A, A, None) == E_SHAPE
    assert f(A, A, 8, A, 2, 128, 0, 0, A + 8, A, A, A, None) == E_ALIGN
    assert f(A, A, 8, A, 2, 128, 2, 0, A, A, A, A, None) == E_ENUM
    assert f(A, A, 8, A, 2, 128, 0, 2, A, A, A, A, None) == E_ENUM
    assert f(A, A, 8, A, 1025, 128, 0, 0, A, A, A, A, None) == E_UNSUP
    assert f(None, None, 0, A, 2, 128, 0, 0, None, None, None, None, None) == OK


@pytest.mark.parametrize("name", ["", "_precise"])
def test_grouped_gemm_rowscaled_refusals(lib, name):
    f = getattr(lib, "fp8q_grouped_gemm_rowscaled" + name)
    assert f(None, A, A, A, 256, A, 2, 128, 128, A, 0, None) == E_NULL
    assert f(A, A, A, A, 256, None, 2, 128, 128, A, 0, None) == E_NULL
    assert f(A, A, A, A, 256, A, 2, 128, 128, None, 0, None) == E_NULL
    assert f(None, None, None, None, 0, A, 2, 128, 128, None, 0, None) == E_NULL
    for bad in ((100, 128, 128), (256, 100, 128), (256, 128, 100), (-128, 128, 128)):
        assert f(A, A, A, A, bad[0], A, 2, bad[1], bad[2], A, 0, None) == E_SHAPE
    assert f(A, A, A, A, 256, A, 0, 128, 128, A, 0, None) == E_SHAPE
    assert f(A + 8, A, A, A, 256, A, 2, 128, 128, A, 0, None) == E_ALIGN
    assert f(A, A, A, A + 2, 256, A, 2, 128, 128, A, 0, None) == E_ALIGN
    assert f(A, A, A, A, 256, A, 2, 128, 128, A, 2, None) == E_ENUM
    assert f(A, A, A, A, 256, A, 1025, 128, 128, A, 0, None) == E_UNSUP
    assert f(A, A, A, A, (1 << 24) + 128, A, 2, 128, 128, A, 0, None) == E_UNSUP
    assert f(None, None, None, None, 256, A, 2, 0, 128, None, 0, None) == OK


def _adamw(lib, tensors=None, count=None, grad=0, moments=0, **kw):
    if tensors is None:
        tensors = [dict()]
    arr = (fq.AdamwTensor * max(1, len(tensors)))()
    for k, t in enumerate(tensors):
        base = A + 4096 * k
        for n, v in {**dict(p=base, g=A, m=A, v=A, m_s=A, v_s=A, n=1024), **t}.items():
            setattr(arr[k], n, v)
    args = fq.AdamwArgs(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)
    for n, v in kw.items():
        setattr(args, n, v)
    return lib.fp8q_adamw(arr, len(tensors) if count is None else count, ctypes.byref(args), grad,
                          moments, None)


def test_adamw_refusals(lib):
    assert lib.fp8q_adamw(None, 1, ctypes.byref(fq.AdamwArgs()), 0, 0, None) == E_NULL
    assert lib.fp8q_adamw(None, 0, None, 0, 0, None) == E_NULL
    for n in "pgmv":
        assert _adamw(lib, [{n: None}]) == E_NULL
        assert _adamw(lib, [{n: A + 8}]) == E_ALIGN
    for n in ("m_s", "v_s"):
        assert _adamw(lib, [{n: None}], moments=1) == E_NULL
        assert _adamw(lib, [{n: A + 2}], moments=1) == E_ALIGN
    assert _adamw(lib, [dict(copy=A + 8)]) == E_ALIGN
    assert _adamw(lib, count=-1) == E_SHAPE
    assert _adamw(lib, [dict(n=-1)]) == E_SHAPE
    assert _adamw(lib, [{}, dict(n=2 ** 34 + 1)], count=2) == E_UNSUP
    for n in ("lr_dev", "step_dev", "grad_scale"):
        assert _adamw(lib, **{n: A + 2}) == E_ALIGN
    assert _adamw(lib, grad=2) == E_ENUM and _adamw(lib, moments=2) == E_ENUM
    nan, inf = float("nan"), float("inf")
    for n in ("lr", "eps", "weight_decay"):
        for v in (-1.0, nan, inf):
            assert _adamw(lib, **{n: v}) == E_UNSUP
    for n in ("beta1", "beta2"):
        for v in (-0.1, 1.0, nan):
            assert _adamw(lib, **{n: v}) == E_UNSUP
    assert _adamw(lib, step=0) == E_UNSUP
    # nothing to do
    assert _adamw(lib, [dict(p=None, g=None, m=None, v=None, n=0)]) == OK
    assert _adamw(lib, [], count=0) == OK


@pytest.mark.parametrize("count", [2, 64, 65, 200])
def test_adamw_refuses_a_tensor_given_twice(lib, count):
    """The same parameter, or an overlapping one, in any two places."""
    for i, j, shift in ((0, count - 1, 0), (count - 1, 0, 0), (0, 1, 0), (count // 2, 0, 1008)):
        t = [dict() for _ in range(count)]
        t[i] = dict(p=A + 4096 * j + 4 * shift)
        if i != j:
            assert _adamw(lib, t) == E_UNSUP, (i, j, shift)


# ------------------------------------------------------------------ the binding
def _t(shape, dt):
    return torch.empty(shape, dtype=dt)


@pytest.fixture
def no_stream():
    with um.patch.object(fq, "_stream", lambda st, d: None):
        yield


def _refuses(fn, good, bad):
    for b in bad:
        with pytest.raises(ValueError):
            fn(**{**good, **b})


def test_binding_refusals_layer_norm(no_stream):
    M, N = 4, 256
    good = dict(x=_t((M, N), bf16), weight=_t((N,), f32), bias=_t((N,), f32), mean=_t((M,), f32),
                rstd=_t((M,), f32), y=_t((M, N), bf16), q=_t((M, N), u8), s=_t((2, M), f32))
    _refuses(fq.fp8q_layer_norm, good,
             [dict(x=_t((M, N), torch.float16)), dict(x=_t((N, M), bf16).t()), dict(x=None),
              dict(weight=_t((N,), bf16)), dict(weight=_t((M,), f32)), dict(bias=_t((N + 1,), f32)),
              dict(mean=_t((N,), f32)), dict(rstd=_t((M, 1), f32)), dict(y=_t((M, N), u8)),
              dict(y=None, q=None, s=None), dict(q=None), dict(s=None), dict(s=_t((M, 2), f32)),
              dict(q=_t((M, N), torch.int8))])
    with pytest.raises(ValueError):
        fq.layer_norm_quantized(_t((M, 200), bf16), _t((200,), f32))
    with pytest.raises(ValueError):
        fq.layer_norm(_t((M, 0), bf16), _t((0,), f32))
    with pytest.raises(ValueError):
        fq.layer_norm(_t((M, 20000), bf16), _t((20000,), f32))
    with pytest.raises(ValueError):
        fq.layer_norm(_t((2, M, N), bf16), _t((N,), f32))
    with pytest.raises(ValueError):
        fq.layer_norm(_t((M, N), bf16), _t((N,), f32), out_dtype=torch.float16)
    M = 64
    work = fq.layer_norm_backward_workspace(M, N)
    good = dict(dy=_t((M, N), bf16), x=_t((M, N), f32), weight=_t((N,), f32), mean=_t((M,), f32),
                rstd=_t((M,), f32), dx=_t((M, N), f32), dweight=_t((N,), f32),
                dbias=_t((N,), f32), workspace=_t((work,), u8))
    _refuses(fq.fp8q_layer_norm_backward, good,
             [dict(dy=_t((M, N), torch.float16)), dict(dy=_t((M + 1, N), bf16)),
              dict(dx=_t((M, N), bf16)), dict(dweight=_t((N,), bf16)), dict(dbias=_t((M,), f32)),
              dict(workspace=_t((work - 1,), u8)), dict(weight=None)])
    with pytest.raises(ValueError):
        fq.layer_norm_backward(_t((M, N), bf16), _t((M, N), f32), _t((M,), f32), _t((M,), f32),
                               _t((M,), f32))


def test_binding_refusals_experts(no_stream):
    M, K, G = 300, 128, 3
    T = fq.expert_columns(M, G)
    off = _t((G + 1,), i32)
    good = dict(x=_t((M, K), bf16), off=off, q_t=_t((K, T), u8), s_t=_t((T // 128, K), f32))
    bad_off = [dict(off=None), dict(off=_t((G + 1,), torch.int64)), dict(off=_t((1,), i32)),
               dict(off=_t((2, 2), i32))]
    _refuses(fq.fp8q_grouped_quantize_act_t, good,
             bad_off + [dict(x=_t((M, K), f32)), dict(q_t=_t((K, M), u8)),
                        dict(s_t=_t((K, T // 128), f32)), dict(x=_t((M, 100), bf16))])
    F = 128
    good = dict(dh=_t((M, F), bf16), gate_up=_t((M, 2 * F), bf16), off=off, q=_t((M, 2 * F), u8),
                s=_t((2, M), f32), qt=_t((2 * F, T), u8), st=_t((T // 128, 2 * F), f32))
    _refuses(fq.fp8q_grouped_gated_backward, good,
             bad_off + [dict(q=None), dict(st=None), dict(q=None, s=None, qt=None, st=None),
                        dict(qt=_t((2 * F, 384), u8)), dict(act="relu"),
                        dict(gate_up=_t((M, F), bf16))])
    N = 256
    good = dict(a_q=_t((N, T), u8), a_s=_t((T // 128, N), f32), b_q=_t((K, T), u8),
                b_s=_t((T // 128, K), f32), off=off, c=_t((G, N, K), bf16))
    for f in (fq.fp8q_grouped_gemm_rowscaled, fq.fp8q_grouped_gemm_rowscaled_precise):
        _refuses(f, good,
                 bad_off + [dict(c=_t((N, K), bf16)), dict(c=_t((G, N, K), torch.float16)),
                            dict(b_q=_t((K, T + 128), u8)), dict(a_s=_t((N, T // 128), f32)),
                            dict(a_q=_t((100, T), u8))])
    with pytest.raises(ValueError):
        fq.grouped_quantize_act_t(_t((M, K), bf16), None)
    with pytest.raises(ValueError):
        fq.grouped_gemm_rowscaled(good["a_q"], good["a_s"], good["b_q"], good["b_s"], off,
                                  out_dtype=torch.float16)
    with pytest.raises(ValueError):
        fq.grouped_gated_backward(_t((M, F), bf16), _t((M, 2 * F), bf16), off, rows=False,
                                  tokens=False)


@pytest.mark.parametrize("eight", [False, True])
def test_binding_refusals_adamw(no_stream, eight):
    n, shape = 3, (5, 60)
    moment = u8 if eight else f32
    good = dict(params=[_t(shape, f32) for _ in range(n)], grads=[_t(shape, bf16) for _ in range(n)],
                exp_avgs=[_t(shape, moment) for _ in range(n)],
                exp_avg_sqs=[_t(shape, moment) for _ in range(n)], step=1)
    fn = fq.adamw
    if eight:
        fn = fq.adamw_8bit
        good.update(exp_avg_scales=[_t((3,), f32) for _ in range(n)],
                    exp_avg_sq_scales=[_t((3,), f32) for _ in range(n)])

    def swap(name, t, at=1):
        l = list(good[name])
        l[at] = t
        return {name: l}
    bad = [swap("params", _t(shape, bf16)), swap("params", None, 0), swap("grads", None),
           swap("grads", None, 0), swap("grads", _t(shape, f32)), swap("grads", _t((60, 5), bf16)),
           swap("grads", _t(shape, torch.float16), 0), swap("exp_avgs", _t((5, 61), moment)),
           swap("exp_avg_sqs", _t(shape, bf16)), swap("params", _t((60, 5), f32).t()),
           dict(copies=[_t(shape, bf16)] * 2), dict(copies=[_t(shape, f32)] * 3),
           dict(step=0), dict(step=_t((1,), torch.int64)), dict(step=_t((2,), i32)),
           dict(lr=-1.0), dict(lr=_t((1,), torch.float64)), dict(betas=(1.0, 0.9)),
           dict(betas=(0.9, -0.1)), dict(eps=-1e-8), dict(weight_decay=float("nan")),
           dict(grad_scale=_t((2,), f32)), dict(grad_scale=1.0), dict(grads=good["grads"][:2])]
    if eight:
        bad += [swap("exp_avg_scales", _t((2,), f32)), swap("exp_avg_sq_scales", _t((3,), bf16))]
    _refuses(fn, good, bad)
    fn(**{k: [] if isinstance(v, list) else v for k, v in good.items()})   # nothing to do
