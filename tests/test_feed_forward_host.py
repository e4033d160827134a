"""The feed-forward calls without a GPU: the oracle's derivatives against
differences, host-side refusals of the C ABI and of the binding."""

import ctypes
import os
import unittest.mock as um

import numpy as np
import pytest
import torch

from oracle import feed_forward as off

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
fq = pytest.importorskip("fine_grained_block_fp8q_amd")

OK, E_NULL, E_SHAPE, E_ALIGN, E_ENUM, E_DEVICE, E_LAUNCH, E_UNSUP, E_OFFSETS = range(9)
u8, i8, f32, bf16, i32 = torch.uint8, torch.int8, torch.float32, torch.bfloat16, torch.int32
A = 0x10000  # a fake aligned address: never dereferenced on these paths


# ------------------------------------------------------------------- the oracle
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_oracle_derivative_against_differences(act):
    """Central differences of step h are off by h^2/6 |f'''| + eps |f| / h: with
    h = 1e-5 and |f'''| below 4 here, under 1e-9 for |x| <= 12."""
    x = np.linspace(-12, 12, 2001)
    h = 1e-5
    d = (off.act(act, x + h) - off.act(act, x - h)) / (2 * h)
    assert np.abs(d - off.act_grad(act, x)).max() < 1e-9


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_oracle_block_gradient_against_differences(act):
    """d/dY of sum(dh * gated(Y)), element by element."""
    rng = np.random.default_rng(3)
    Y, dh = rng.standard_normal((3, 8)) * 2, rng.standard_normal((3, 4))
    got = off.gated_backward(act, dh, Y)
    h = 1e-5
    for i in range(3):
        for j in range(8):
            p, m = Y.copy(), Y.copy()
            p[i, j] += h
            m[i, j] -= h
            d = ((dh * off.gated(act, p)).sum() - (dh * off.gated(act, m)).sum()) / (2 * h)
            assert abs(d - got[i, j]) < 1e-8


def test_oracle_activations_known_values():
    assert off.act("silu", 0.0) == 0 and off.act_grad("silu", 0.0) == 0.5
    assert off.act("gelu_tanh", 0.0) == 0 and off.act_grad("gelu_tanh", 0.0) == 0.5
    assert abs(off.act("silu", 1.0) - 1 / (1 + np.exp(-1.0))) < 1e-15
    x = 1.5
    t = np.tanh(np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3))
    assert abs(off.act("gelu_tanh", x) - 0.5 * x * (1 + t)) < 1e-15


# -------------------------------------------------------------------- the C ABI
@pytest.fixture(params=["libfp8q.so", "libfp8q_debug.so"])
def lib(request):
    L = ctypes.CDLL(os.path.join(ROOT, "fine_grained_block_fp8q_amd", request.param))
    for n in ("fp8q_quantize_token_i8", "fp8q_gemm_i8", "fp8q_gemm_i8_gated", "fp8q_gemm_gated",
              "fp8q_grouped_gemm_gated", "fp8q_gated_backward"):
        getattr(L, n).argtypes = getattr(fq.lib, n).argtypes
    return L


def test_quantize_token_i8_refusals(lib):
    f = lib.fp8q_quantize_token_i8
    assert f(None, 4, 100, A, A, None) == E_NULL
    assert f(A, 4, 100, None, A, None) == E_NULL
    assert f(A, 4, 100, A, None, None) == E_NULL
    assert f(None, 0, 100, None, None, None) == OK
    assert f(A, -1, 100, A, A, None) == E_SHAPE
    assert f(A, 4, -1, A, A, None) == E_SHAPE
    assert f(A + 2, 4, 100, A, A, None) == E_ALIGN
    assert f(A, 4, 100, A + 8, A, None) == E_ALIGN
    assert f(A, 4, 100, A, A + 2, None) == E_ALIGN
    assert f(A, 4, 0, A, A, None) == E_UNSUP


def test_gemm_i8_refusals(lib):
    f = lib.fp8q_gemm_i8
    assert f(None, A, A, A, None, 4, 5, 32, A, 0, None) == E_NULL
    assert f(A, A, A, A, None, 4, 5, 32, None, 0, None) == E_NULL
    assert f(A, A, A, None, None, 4, 5, 32, A, 0, None) == E_NULL
    assert f(A, A, A, A, None, 4, 5, 40, A, 0, None) == E_SHAPE
    assert f(A, A, A, A, None, -4, 5, 32, A, 0, None) == E_SHAPE
    assert f(A, A, A, A, None, 4, -5, 32, A, 0, None) == E_SHAPE
    assert f(A + 8, A, A, A, None, 4, 5, 32, A, 0, None) == E_ALIGN
    assert f(A, A, A, A, A + 1, 4, 5, 32, A, 0, None) == E_ALIGN
    assert f(A, A, A, A, None, 4, 5, 32, A + 4, 0, None) == E_ALIGN
    assert f(A, A, A, A, None, 4, 5, 32, A, 2, None) == E_ENUM
    assert f(None, None, None, None, None, 0, 5, 32, None, 0, None) == OK
    assert f(None, None, None, None, None, 4, 0, 32, None, 0, None) == OK
    assert f(A, A, A, A, None, 4, 5, 0, A, 0, None) == E_UNSUP
    assert f(A, A, A, A, None, 4, 5, 131072, A, 0, None) == E_UNSUP  # the sum could leave int32


def test_gemm_i8_gated_refusals(lib):
    f = lib.fp8q_gemm_i8_gated
    assert f(A, A, None, A, 4, 5, 32, 0, A, 1, None) == E_NULL
    assert f(A, A, A, A, 4, 5, 24, 0, A, 1, None) == E_SHAPE
    assert f(A, A, A + 1, A, 4, 5, 32, 0, A, 1, None) == E_ALIGN
    assert f(A, A, A, A, 4, 5, 32, 2, A, 1, None) == E_ENUM
    assert f(A, A, A, A, 4, 5, 32, 0, A, 3, None) == E_ENUM
    assert f(A, A, A, A, 4, 5, 131072, 0, A, 1, None) == E_UNSUP
    assert f(None, None, None, None, 0, 5, 32, 0, None, 1, None) == OK


def test_gemm_gated_refusals(lib):
    f = lib.fp8q_gemm_gated
    assert f(None, A, A, A, 4, 128, 128, 0, A, 1, None, None) == E_NULL
    assert f(A, A, A, A, 4, 128, 128, 0, None, 1, A, None) == E_NULL
    assert f(A, A, A, A, 4, 64, 128, 0, A, 1, None, None) == E_SHAPE
    assert f(A, A, A, A, 4, 128, 64, 0, A, 1, None, None) == E_SHAPE
    assert f(A, A, A, A, 4, 128, 128, 0, A, 1, A + 2, None) == E_ALIGN
    assert f(A, A, A, A, 4, 128, 128, 5, A, 1, None, None) == E_ENUM
    assert f(A, A, A, A, 4, 128, 128, 0, A, 5, None, None) == E_ENUM
    assert f(A, A, A, A, 4, 128, 0, 0, A, 1, None, None) == E_UNSUP
    assert f(A, A, A, A, 4, 128, (1 << 22) + 128, 0, A, 1, None, None) == E_UNSUP
    assert f(None, None, None, None, 0, 128, 128, 0, None, 1, None, None) == OK


def test_grouped_gemm_gated_refusals(lib):
    f = lib.fp8q_grouped_gemm_gated
    assert f(A, A, 8, None, 2, A, A, 128, 128, 0, A, 1, None, None) == E_NULL
    assert f(A, A, 8, A, 2, A, A, 128, 128, 0, None, 1, None, None) == E_NULL
    assert f(A, A, 8, A, 0, A, A, 128, 128, 0, A, 1, None, None) == E_SHAPE
    assert f(A, A, 1 << 31, A, 2, A, A, 128, 128, 0, A, 1, None, None) == E_SHAPE
    assert f(A, A, 8, A + 2, 2, A, A, 128, 128, 0, A, 1, None, None) == E_ALIGN
    assert f(A, A, 8, A, 2, A, A, 128, 128, 9, A, 1, None, None) == E_ENUM
    assert f(A, A, 8, A, 2000, A, A, 128, 128, 0, A, 1, None, None) == E_UNSUP
    assert f(None, None, 0, A, 2, None, None, 128, 128, 0, None, 1, None, None) == OK


def test_gated_backward_refusals(lib):
    f = lib.fp8q_gated_backward
    assert f(None, A, 4, 128, 0, 0, A, A, A, A, None) == E_NULL
    assert f(A, A, 4, 128, 0, 0, A, None, A, A, None) == E_NULL
    assert f(A, A, 4, 128, 0, 0, A, A, None, A, None) == E_NULL
    assert f(A, A, 4, 128, 0, 0, None, None, None, None, None) == E_NULL
    assert f(A, A, 4, 100, 0, 0, A, A, A, A, None) == E_SHAPE
    assert f(A, A, -4, 128, 0, 0, A, A, A, A, None) == E_SHAPE
    assert f(A, A + 8, 4, 128, 0, 0, A, A, A, A, None) == E_ALIGN
    assert f(A, A, 4, 128, 0, 0, A, A + 2, None, None, None) == E_ALIGN
    assert f(A, A, 4, 128, 2, 0, A, A, A, A, None) == E_ENUM
    assert f(A, A, 4, 128, 0, 2, A, A, A, A, None) == E_ENUM
    assert f(None, None, 0, 128, 0, 0, None, None, None, None, None) == OK
    assert f(A, A, 4, (1 << 22) + 128, 0, 0, A, A, A, A, None) == E_UNSUP


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


def test_binding_refusals_i8(no_stream):
    _refuses(fq.fp8q_quantize_token_i8,
             dict(x=_t((4, 100), bf16), q=_t((4, 112), i8), s=_t((4,), f32)),
             [dict(x=_t((4, 100), f32)), dict(q=_t((4, 100), i8)), dict(q=_t((4, 112), u8)),
              dict(s=_t((5,), f32)), dict(x=_t((100, 4), bf16).t())])
    good = dict(a_q=_t((4, 64), i8), a_s=_t((4,), f32), w_q=_t((10, 64), i8), w_s=_t((10,), f32),
                c=_t((4, 10), bf16), bias=_t((10,), f32))
    _refuses(fq.fp8q_gemm_i8, good,
             [dict(a_q=_t((4, 64), u8)), dict(a_s=_t((1, 4), f32)), dict(w_q=_t((10, 80), i8)),
              dict(w_s=_t((9,), f32)), dict(c=_t((4, 10), torch.float16)), dict(c=_t((4, 11), bf16)),
              dict(bias=_t((10,), bf16)), dict(bias=_t((11,), f32)),
              dict(a_q=_t((4, 60), i8), w_q=_t((10, 60), i8))])
    good = dict(a_q=_t((4, 64), i8), a_s=_t((4,), f32), w_q=_t((10, 64), i8), w_s=_t((10,), f32),
                h=_t((4, 5), bf16))
    _refuses(fq.fp8q_gemm_i8_gated, good,
             [dict(w_q=_t((9, 64), i8), w_s=_t((9,), f32)), dict(h=_t((4, 10), bf16)),
              dict(act="relu")])


def test_binding_refusals_gated(no_stream):
    M, F, K = 5, 128, 256
    good = dict(a_q=_t((M, K), u8), a_s=_t((2, M), f32), w_q=_t((2 * F, K), u8),
                w_s=_t((2, 2), f32), h=_t((M, F), bf16), gate_up=_t((M, 2 * F), bf16))
    bad = [dict(h=_t((M, 2 * F), bf16)), dict(gate_up=_t((M, 2 * F), f32)),
           dict(gate_up=_t((M, F), bf16)), dict(act="tanh"), dict(w_s=_t((1, 2), f32)),
           dict(a_q=_t((M, K), i8)), dict(h=_t((M, F), torch.float16))]
    _refuses(fq.fp8q_gemm_gated, good, bad + [dict(w_q=_t((3 * 128, K), u8), w_s=_t((3, 2), f32))])
    G = 3
    good.update(off=_t((G + 1,), i32), w_q=_t((G, 2 * F, K), u8), w_s=_t((G, 2, 2), f32))
    _refuses(fq.fp8q_grouped_gemm_gated, good,
             bad + [dict(off=_t((G,), i32)), dict(off=_t((G + 1,), torch.int64)),
                    dict(off=None)])


def test_binding_refusals_backward(no_stream):
    M, F = 5, 128
    good = dict(dh=_t((M, F), bf16), gate_up=_t((M, 2 * F), bf16), q=_t((M, 2 * F), u8),
                s=_t((2, M), f32), qt=_t((2 * F, 128), u8), st=_t((1, 2 * F), f32))
    _refuses(fq.fp8q_gated_backward, good,
             [dict(dh=_t((M, F), f32)), dict(gate_up=_t((M, F), bf16)), dict(q=None),
              dict(q=None, s=None, qt=None, st=None), dict(qt=_t((2 * F, M), u8)),
              dict(st=_t((2, 2 * F), f32)), dict(s=_t((M, 2), f32)), dict(act="relu"),
              dict(dh=_t((M, 100), bf16), gate_up=_t((M, 200), bf16))])


def test_allocating_calls_refuse_as_the_wrappers_do(no_stream):
    """Arguments the compiled path does not take reach the wrappers' checks."""
    a, s, w, ws = _t((4, 64), i8), _t((4,), f32), _t((10, 64), i8), _t((10,), f32)
    for args, kw in (((a, s, _t((10, 80), i8), ws), {}), ((a, s[:2], w, ws), {}),
                     ((a, s, w, ws), dict(out_dtype=torch.float16)),
                     ((a, s, w, ws), dict(bias=_t((9,), f32))), ((None, s, w, ws), {})):
        with pytest.raises(ValueError):
            fq.gemm_i8(*args, **kw)
    with pytest.raises(ValueError):
        fq.gemm_i8_gated(a, s, w[:9], ws[:9])
    with pytest.raises(ValueError):
        fq.gemm_i8_gated(a, s, w, ws, act="relu")
    with pytest.raises(ValueError):
        fq.quantize_token_i8(_t((4, 64), f32))
    with pytest.raises(ValueError):
        fq.gemm_gated(_t((4, 128), u8), _t((1, 4), f32), _t((128, 128), u8), _t((1, 1), f32))
    with pytest.raises(ValueError):
        fq.grouped_gemm_gated(_t((4, 128), u8), _t((1, 4), f32), None, _t((2, 256, 128), u8),
                              _t((2, 2, 1), f32))
    with pytest.raises(ValueError):
        fq.gated_backward(_t((4, 128), bf16), _t((4, 256), bf16), rows=False, tokens=False)
    with pytest.raises(ValueError):
        fq.gated_backward(_t((4, 128), bf16), _t((4, 128), bf16))
