"""Python binding of libfp8q (MI355X / gfx950 fine-grained block-scaled FP8).

Argument marshalling only: each function below has the name of the C entry
point it wraps (include/fp8q.h), takes torch tensors, passes their device
pointers, sizes and the current HIP stream, and raises Fp8qError on a non-OK
status.  Every step of the computation runs in the HIP kernels of
libfp8q.so; there is no fallback path -- importing this package without the
built library raises ImportError.

Before each call the wrappers check on the host what the C ABI cannot see
(raising ValueError): every tensor's dtype, contiguity and device, and that
the operand, scale, offset and output shapes agree with each other.  The C
library then validates sizes, alignment and enums itself.

Allocation helpers (``quantize_act``, ``quantize_weight``, ``gemm``,
``grouped_gemm``, ...) allocate outputs with torch on the input's device and
then call the entry points.  Given a ``stream``, they allocate on it; the caller
orders the inputs before the call and its own use of the outputs behind it, and
keeps the inputs until it has run (the outputs may be dropped at any time).  Those of the feed-forward operators and of a
training step (``quantize_token_i8``, ``gemm_i8``, ``gemm_gated``, ...;
``layer_norm``, ``grouped_gemm_rowscaled``, ``adamw``, ...) do so in compiled code
(csrc/calls.cpp) when every argument is as it should be and no stream is named;
else, and where the compiled module cannot be loaded, they take the Python path,
whose checks say what is wrong.
"""

import ctypes
import os
import warnings
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8q.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libfp8q.so not found at {LIB_PATH}; build it with "
        "`python fine_grained_block_fp8q_amd/build.py` (hipcc, gfx950)")

lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_st = ctypes.c_int

lib.fp8q_quantize_act.argtypes = [_p, _i64, _i64, _p, _p, _i32, _p]
lib.fp8q_quantize_act.restype = _st
lib.fp8q_quantize_weight.argtypes = [_p, _i64, _i64, _p, _p, _i32, _p]
lib.fp8q_quantize_weight.restype = _st
lib.fp8q_gemm.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _p, _i32, _p]
lib.fp8q_gemm.restype = _st
lib.fp8q_gemm_precise.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _p, _i32, _p]
lib.fp8q_gemm_precise.restype = _st
lib.fp8q_gemm_mfma_scaled.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _p, _i32, _p]
lib.fp8q_gemm_mfma_scaled.restype = _st
lib.fp8q_grouped_gemm.argtypes = [_p, _p, _i64, _p, _i32, _p, _p, _i64, _i64, _p, _i32, _p]
lib.fp8q_grouped_gemm.restype = _st
lib.fp8q_grouped_gemm_precise.argtypes = [_p, _p, _i64, _p, _i32, _p, _p, _i64, _i64, _p, _i32,
                                          _p]
lib.fp8q_grouped_gemm_precise.restype = _st
lib.fp8q_gemm_bf16.argtypes = [_p, _p, _i64, _i64, _i64, _p, _i32, _p]
lib.fp8q_quantize_act_t.argtypes = [_p, _i64, _i64, _p, _p, _i32, _p]
lib.fp8q_quantize_act_t.restype = _st
lib.fp8q_quantize_weight_t.argtypes = [_p, _i64, _i64, _p, _p, _i32, _p]
lib.fp8q_quantize_weight_t.restype = _st
lib.fp8q_gemm_rowscaled.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _p, _i32, _p]
lib.fp8q_gemm_rowscaled.restype = _st
lib.fp8q_gemm_rowscaled_precise.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _p, _i32, _p]
lib.fp8q_gemm_rowscaled_precise.restype = _st
lib.fp8q_gemm_bf16.restype = _st
lib.fp8q_gemm_fused.argtypes = [_p, _p, _p, _i64, _i64, _i64, _p, _i32, _i32, _p]
lib.fp8q_gemm_fused.restype = _st
lib.fp8q_grouped_gemm_fused.argtypes = [_p, _i64, _p, _i32, _p, _p, _i64, _i64, _p, _i32, _i32,
                                        _p]
lib.fp8q_grouped_gemm_fused.restype = _st
lib.fp8q_quantize_token_i8.argtypes = [_p, _i64, _i64, _p, _p, _p]
lib.fp8q_quantize_token_i8.restype = _st
lib.fp8q_gemm_i8.argtypes = [_p, _p, _p, _p, _p, _i64, _i64, _i64, _p, _i32, _p]
lib.fp8q_gemm_i8.restype = _st
lib.fp8q_gemm_i8_gated.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _i32, _p, _i32, _p]
lib.fp8q_gemm_i8_gated.restype = _st
lib.fp8q_gemm_gated.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _i32, _p, _i32, _p, _p]
lib.fp8q_gemm_gated.restype = _st
lib.fp8q_grouped_gemm_gated.argtypes = [_p, _p, _i64, _p, _i32, _p, _p, _i64, _i64, _i32, _p, _i32,
                                        _p, _p]
lib.fp8q_grouped_gemm_gated.restype = _st
lib.fp8q_gated_backward.argtypes = [_p, _p, _i64, _i64, _i32, _i32, _p, _p, _p, _p, _p]
lib.fp8q_gated_backward.restype = _st
_f32 = ctypes.c_float
lib.fp8q_layer_norm.argtypes = [_p, _i32, _p, _p, _i64, _i64, _f32, _p, _i32, _p, _p, _i32, _p, _p,
                                _p]
lib.fp8q_layer_norm.restype = _st
lib.fp8q_layer_norm_backward_workspace.argtypes = [_i64, _i64]
lib.fp8q_layer_norm_backward_workspace.restype = _i64
lib.fp8q_layer_norm_backward.argtypes = [_p, _i32, _p, _i32, _p, _p, _p, _i64, _i64, _p, _p, _p,
                                         _p, _p]
lib.fp8q_layer_norm_backward.restype = _st
lib.fp8q_expert_columns.argtypes = [_i64, _i32]
lib.fp8q_expert_columns.restype = _i64
lib.fp8q_grouped_quantize_act_t.argtypes = [_p, _i64, _p, _i32, _i64, _p, _p, _i32, _p]
lib.fp8q_grouped_quantize_act_t.restype = _st
lib.fp8q_grouped_gated_backward.argtypes = [_p, _p, _i64, _p, _i32, _i64, _i32, _i32, _p, _p, _p,
                                            _p, _p]
lib.fp8q_grouped_gated_backward.restype = _st
lib.fp8q_grouped_gemm_rowscaled.argtypes = [_p, _p, _p, _p, _i64, _p, _i32, _i64, _i64, _p, _i32,
                                            _p]
lib.fp8q_grouped_gemm_rowscaled.restype = _st
lib.fp8q_grouped_gemm_rowscaled_precise.argtypes = lib.fp8q_grouped_gemm_rowscaled.argtypes
lib.fp8q_grouped_gemm_rowscaled_precise.restype = _st


class AdamwTensor(ctypes.Structure):
    """fp8q_adamw_tensor"""
    _fields_ = [("p", _p), ("g", _p), ("m", _p), ("v", _p), ("m_s", _p), ("v_s", _p), ("copy", _p),
                ("n", _i64)]


class AdamwArgs(ctypes.Structure):
    """fp8q_adamw_args"""
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + \
               [("step", _i64), ("lr_dev", _p), ("step_dev", _p), ("grad_scale", _p)]


lib.fp8q_adamw.argtypes = [ctypes.POINTER(AdamwTensor), _i32, ctypes.POINTER(AdamwArgs), _i32, _i32,
                           _p]
lib.fp8q_adamw.restype = _st
lib.fp8q_status_string.argtypes = [_st]
lib.fp8q_status_string.restype = ctypes.c_char_p
lib.fp8q_abi_version.argtypes = []
lib.fp8q_abi_version.restype = ctypes.c_int
lib.fp8q_debug_checks.argtypes = []
lib.fp8q_debug_checks.restype = ctypes.c_int

# enums (include/fp8q.h)
(OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ENUM, ERR_DEVICE, ERR_LAUNCH, ERR_UNSUPPORTED,
 ERR_OFFSETS) = range(9)
SCALE_F32, SCALE_POW2 = 0, 1
OUT_F32, OUT_BF16 = 0, 1
ACT_SILU, ACT_GELU_TANH = 0, 1
MOMENTS_F32, MOMENTS_E4M3 = 0, 1
GROUP = 128

_MODES = {"f32": SCALE_F32, "pow2": SCALE_POW2, SCALE_F32: SCALE_F32, SCALE_POW2: SCALE_POW2}
_OUTS = {"f32": OUT_F32, "bf16": OUT_BF16, OUT_F32: OUT_F32, OUT_BF16: OUT_BF16}
_ACTS = {"silu": ACT_SILU, "gelu_tanh": ACT_GELU_TANH, ACT_SILU: ACT_SILU,
         ACT_GELU_TANH: ACT_GELU_TANH}


class Fp8qError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {lib.fp8q_status_string(status).decode()}")


def _check(status, where):
    if status != OK:
        raise Fp8qError(status, where)


class _Bound(Exception):
    """Raised inside a wrapper called through bind(): carries the C call."""

    def __init__(self, call):
        super().__init__("bound call")
        self.call = call


_capture = threading.local()


def _invoke(cfunc, args, where, updated=()):
    """`updated`: tensors that the call changes in place, of which autograd is to hear."""
    if getattr(_capture, "on", False):
        raise _Bound((cfunc, args, where, updated))
    _check(cfunc(*args), where)
    _bumped(updated)


def _bumped(tensors):
    """Tells autograd that these were written."""
    if tensors:
        import torch
        torch.autograd.graph.increment_version([t for t in tensors if not t.is_inference()])


def bind(fn, *args, **kwargs):
    """Validate a call once and return a zero-argument callable that repeats
    it: the same C entry point with the same pointers, sizes and stream, and
    none of the per-call host checks (for launch loops whose kernels are
    shorter than those checks).  The callable holds references to the
    arguments, so their tensors stay alive while it exists; they must keep
    their storage (no resize or set_) while it is used.  A non-OK status
    still raises.  Example: run = bind(fp8q_quantize_act, x, q, s); run(); run()."""
    _capture.on = True
    try:
        fn(*args, **kwargs)
    except _Bound as b:
        cfunc, cargs, where, updated = b.call
    else:
        raise TypeError(f"{getattr(fn, '__name__', fn)} is not an entry-point wrapper")
    finally:
        _capture.on = False

    # the pointers in cargs refer to these tensors' storage (a list may change later)
    own = lambda a: tuple(a) if isinstance(a, list) else a   # noqa: E731
    keep = (tuple(own(a) for a in args), {k: own(a) for k, a in kwargs.items()})

    def run():
        st = cfunc(*cargs)
        if st != OK:
            raise Fp8qError(st, where)
        _bumped(updated)
    run.args = keep
    return run


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_DTYPES = {"u8": "uint8", "f32": "float32", "bf16": "bfloat16", "i32": "int32", "i8": "int8"}


def _dt(name):
    import torch
    return getattr(torch, _DTYPES[name])


def _req(where, name, t, dtypes, shape, device):
    """Host-side check of one tensor argument: dtype, contiguity, device, shape."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{where}: {name} must be a torch.Tensor")
    allowed = [_dt(d) for d in dtypes]
    if t.dtype not in allowed:
        raise ValueError(f"{where}: {name} has dtype {t.dtype}, expected one of {allowed}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{where}: {name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dims(where, t, ndim, name):
    import torch
    if not isinstance(t, torch.Tensor) or t.dim() != ndim:
        raise ValueError(f"{where}: {name} must be a {ndim}-d torch.Tensor")
    return t.shape


def _mult128(where, **dims):
    for k, v in dims.items():
        if v % GROUP:
            raise ValueError(f"{where}: {k} = {v} is not a multiple of {GROUP}")


def _out_code(where, c):
    import torch
    if c.dtype == torch.bfloat16:
        return OUT_BF16
    if c.dtype == torch.float32:
        return OUT_F32
    raise ValueError(f"{where}: c has dtype {c.dtype}, expected float32 or bfloat16")


def _stream(stream, device):
    import torch
    if stream is None:
        if device.type == "cuda":     # the handle alone, without a Stream object around it
            return torch._C._cuda_getCurrentRawStream(device.index)
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def abi_version():
    return lib.fp8q_abi_version()


# ---------------------------------------------------------------- entry points
def fp8q_quantize_act(x, q, s, mode="f32", stream=None):
    """x: bf16 [M][K] -> q: uint8 [M][K], s: float32 [K/128][M] (in place)."""
    w = "fp8q_quantize_act"
    M, K = _dims(w, x, 2, "x")
    _mult128(w, K=K)
    _req(w, "x", x, ["bf16"], (M, K), x.device)
    _req(w, "q", q, ["u8"], (M, K), x.device)
    _req(w, "s", s, ["f32"], (K // GROUP, M), x.device)
    _invoke(lib.fp8q_quantize_act, (_ptr(x), M, K, _ptr(q), _ptr(s), _MODES[mode],
                                 _stream(stream, x.device)), "fp8q_quantize_act")


def fp8q_quantize_weight(w, q, s, mode="f32", stream=None):
    """w: bf16 [N][K] -> q: uint8 [N][K], s: float32 [N/128][K/128] (in place)."""
    wh = "fp8q_quantize_weight"
    N, K = _dims(wh, w, 2, "w")
    _mult128(wh, N=N, K=K)
    _req(wh, "w", w, ["bf16"], (N, K), w.device)
    _req(wh, "q", q, ["u8"], (N, K), w.device)
    _req(wh, "s", s, ["f32"], (N // GROUP, K // GROUP), w.device)
    _invoke(lib.fp8q_quantize_weight, (_ptr(w), N, K, _ptr(q), _ptr(s), _MODES[mode],
                                    _stream(stream, w.device)), "fp8q_quantize_weight")


def _gemm_args(where, a_q, a_s, w_q, w_s, c):
    M, K = _dims(where, a_q, 2, "a_q")
    N, _ = _dims(where, w_q, 2, "w_q")
    _mult128(where, N=N, K=K)
    dev = a_q.device
    _req(where, "a_q", a_q, ["u8"], (M, K), dev)
    _req(where, "a_s", a_s, ["f32"], (K // GROUP, M), dev)
    _req(where, "w_q", w_q, ["u8"], (N, K), dev)
    _req(where, "w_s", w_s, ["f32"], (N // GROUP, K // GROUP), dev)
    _req(where, "c", c, ["f32", "bf16"], (M, N), dev)
    return M, N, K, _out_code(where, c)


def fp8q_gemm(a_q, a_s, w_q, w_s, c, stream=None):
    """c[M][N] (float32 or bfloat16) = block-scaled a_q[M][K] x w_q[N][K]^T."""
    M, N, K, out = _gemm_args("fp8q_gemm", a_q, a_s, w_q, w_s, c)
    _invoke(lib.fp8q_gemm, (_ptr(a_q), _ptr(a_s), _ptr(w_q), _ptr(w_s), M, N, K, _ptr(c), out,
                         _stream(stream, a_q.device)), "fp8q_gemm")


def fp8q_gemm_precise(a_q, a_s, w_q, w_s, c, stream=None):
    """fp8q_gemm with each chunk partial formed by FP16 MFMAs on the widened codes."""
    M, N, K, out = _gemm_args("fp8q_gemm_precise", a_q, a_s, w_q, w_s, c)
    _invoke(lib.fp8q_gemm_precise, (_ptr(a_q), _ptr(a_s), _ptr(w_q), _ptr(w_s), M, N, K, _ptr(c),
                                 out, _stream(stream, a_q.device)), "fp8q_gemm_precise")


def fp8q_gemm_mfma_scaled(a_q, a_s, w_q, w_s, c, stream=None):
    """fp8q_gemm with power-of-two scales applied by the matrix core (E8M0)."""
    M, N, K, out = _gemm_args("fp8q_gemm_mfma_scaled", a_q, a_s, w_q, w_s, c)
    _invoke(lib.fp8q_gemm_mfma_scaled, (_ptr(a_q), _ptr(a_s), _ptr(w_q), _ptr(w_s), M, N, K,
                                     _ptr(c), out, _stream(stream, a_q.device)),
            "fp8q_gemm_mfma_scaled")


def _grouped_args(where, a_q, a_s, off, w_q, w_s, c):
    M_total, K = _dims(where, a_q, 2, "a_q")
    G, N, _ = _dims(where, w_q, 3, "w_q")
    _mult128(where, N=N, K=K)
    dev = a_q.device
    _req(where, "a_q", a_q, ["u8"], (M_total, K), dev)
    _req(where, "a_s", a_s, ["f32"], (K // GROUP, M_total), dev)
    _req(where, "off", off, ["i32"], (G + 1,), dev)
    _req(where, "w_q", w_q, ["u8"], (G, N, K), dev)
    _req(where, "w_s", w_s, ["f32"], (G, N // GROUP, K // GROUP), dev)
    _req(where, "c", c, ["f32", "bf16"], (M_total, N), dev)
    return M_total, G, N, K, _out_code(where, c)


def fp8q_grouped_gemm(a_q, a_s, off, w_q, w_s, c, stream=None):
    """Rows [off[e], off[e+1]) of a_q times expert e's w_q[e]; off is a device int32[G+1]."""
    M_total, G, N, K, out = _grouped_args("fp8q_grouped_gemm", a_q, a_s, off, w_q, w_s, c)
    _invoke(lib.fp8q_grouped_gemm, (_ptr(a_q), _ptr(a_s), M_total, _ptr(off), G, _ptr(w_q),
                                 _ptr(w_s), N, K, _ptr(c), out, _stream(stream, a_q.device)), "fp8q_grouped_gemm")


def fp8q_grouped_gemm_precise(a_q, a_s, off, w_q, w_s, c, stream=None):
    """fp8q_grouped_gemm in the precise mode (FP16 MFMAs on the widened codes)."""
    M_total, G, N, K, out = _grouped_args("fp8q_grouped_gemm_precise", a_q, a_s, off, w_q, w_s,
                                          c)
    _invoke(lib.fp8q_grouped_gemm_precise, (_ptr(a_q), _ptr(a_s), M_total, _ptr(off), G, _ptr(w_q),
                                         _ptr(w_s), N, K, _ptr(c), out,
                                         _stream(stream, a_q.device)), "fp8q_grouped_gemm_precise")


def fp8q_gemm_fused(x, w_q, w_s, c, mode="f32", stream=None):
    """c[M][N] = fp8q_gemm(quantize_act(x, mode), w_q, w_s), x: bf16 [M][K]
    quantized inside the GEMM."""
    wh = "fp8q_gemm_fused"
    M, K = _dims(wh, x, 2, "x")
    N, _ = _dims(wh, w_q, 2, "w_q")
    _mult128(wh, N=N, K=K)
    _req(wh, "x", x, ["bf16"], (M, K), x.device)
    _req(wh, "w_q", w_q, ["u8"], (N, K), x.device)
    _req(wh, "w_s", w_s, ["f32"], (N // GROUP, K // GROUP), x.device)
    _req(wh, "c", c, ["f32", "bf16"], (M, N), x.device)
    out = _out_code(wh, c)
    _invoke(lib.fp8q_gemm_fused, (_ptr(x), _ptr(w_q), _ptr(w_s), M, N, K, _ptr(c), out,
                               _MODES[mode], _stream(stream, x.device)), "fp8q_gemm_fused")


def fp8q_grouped_gemm_fused(x, off, w_q, w_s, c, mode="f32", stream=None):
    """The grouped GEMM of quantize_act(x, mode), x: bf16 [M_total][K]
    quantized inside the GEMM; off is a device int32[G+1]."""
    wh = "fp8q_grouped_gemm_fused"
    M_total, K = _dims(wh, x, 2, "x")
    G, N, _ = _dims(wh, w_q, 3, "w_q")
    _mult128(wh, N=N, K=K)
    _req(wh, "x", x, ["bf16"], (M_total, K), x.device)
    _req(wh, "off", off, ["i32"], (G + 1,), x.device)
    _req(wh, "w_q", w_q, ["u8"], (G, N, K), x.device)
    _req(wh, "w_s", w_s, ["f32"], (G, N // GROUP, K // GROUP), x.device)
    _req(wh, "c", c, ["f32", "bf16"], (M_total, N), x.device)
    out = _out_code(wh, c)
    _invoke(lib.fp8q_grouped_gemm_fused, (_ptr(x), M_total, _ptr(off), G, _ptr(w_q), _ptr(w_s), N,
                                       K, _ptr(c), out, _MODES[mode],
                                       _stream(stream, x.device)), "fp8q_grouped_gemm_fused")


def fp8q_gemm_bf16(a, w, c, stream=None):
    """c[M][N] (float32 or bfloat16) = a[M][K] x w[N][K]^T, BF16 operands."""
    wh = "fp8q_gemm_bf16"
    M, K = _dims(wh, a, 2, "a")
    N, _ = _dims(wh, w, 2, "w")
    _mult128(wh, N=N, K=K)
    _req(wh, "a", a, ["bf16"], (M, K), a.device)
    _req(wh, "w", w, ["bf16"], (N, K), a.device)
    _req(wh, "c", c, ["f32", "bf16"], (M, N), a.device)
    out = _out_code(wh, c)
    _invoke(lib.fp8q_gemm_bf16, (_ptr(a), _ptr(w), M, N, K, _ptr(c), out, _stream(stream, a.device)), "fp8q_gemm_bf16")


def fp8q_quantize_act_t(x, q_t, s_t, mode="f32", stream=None):
    """x: bf16 [M][K] -> q_t: uint8 [K][M], s_t: float32 [M/128][K] (in place)."""
    wh = "fp8q_quantize_act_t"
    M, K = _dims(wh, x, 2, "x")
    _mult128(wh, M=M, K=K)
    _req(wh, "x", x, ["bf16"], (M, K), x.device)
    _req(wh, "q_t", q_t, ["u8"], (K, M), x.device)
    _req(wh, "s_t", s_t, ["f32"], (M // GROUP, K), x.device)
    _invoke(lib.fp8q_quantize_act_t, (_ptr(x), M, K, _ptr(q_t), _ptr(s_t), _MODES[mode],
                                   _stream(stream, x.device)), "fp8q_quantize_act_t")


def fp8q_quantize_weight_t(w, q_t, s_t, mode="f32", stream=None):
    """w: bf16 [N][K] -> q_t: uint8 [K][N], s_t: float32 [K/128][N/128] (in place)."""
    wh = "fp8q_quantize_weight_t"
    N, K = _dims(wh, w, 2, "w")
    _mult128(wh, N=N, K=K)
    _req(wh, "w", w, ["bf16"], (N, K), w.device)
    _req(wh, "q_t", q_t, ["u8"], (K, N), w.device)
    _req(wh, "s_t", s_t, ["f32"], (K // GROUP, N // GROUP), w.device)
    _invoke(lib.fp8q_quantize_weight_t, (_ptr(w), N, K, _ptr(q_t), _ptr(s_t), _MODES[mode],
                                      _stream(stream, w.device)), "fp8q_quantize_weight_t")


def _rowscaled_args(where, a_q, a_s, b_q, b_s, c):
    M, K = _dims(where, a_q, 2, "a_q")
    N, _ = _dims(where, b_q, 2, "b_q")
    _mult128(where, N=N, K=K)
    dev = a_q.device
    _req(where, "a_q", a_q, ["u8"], (M, K), dev)
    _req(where, "a_s", a_s, ["f32"], (K // GROUP, M), dev)
    _req(where, "b_q", b_q, ["u8"], (N, K), dev)
    _req(where, "b_s", b_s, ["f32"], (K // GROUP, N), dev)
    _req(where, "c", c, ["f32", "bf16"], (M, N), dev)
    return M, N, K, _out_code(where, c)


def fp8q_gemm_rowscaled(a_q, a_s, b_q, b_s, c, stream=None):
    """c[M][N] = a_q[M][K] x b_q[N][K]^T with 1x128 row-group scales on both."""
    M, N, K, out = _rowscaled_args("fp8q_gemm_rowscaled", a_q, a_s, b_q, b_s, c)
    _invoke(lib.fp8q_gemm_rowscaled, (_ptr(a_q), _ptr(a_s), _ptr(b_q), _ptr(b_s), M, N, K, _ptr(c),
                                   out, _stream(stream, a_q.device)), "fp8q_gemm_rowscaled")


def fp8q_gemm_rowscaled_precise(a_q, a_s, b_q, b_s, c, stream=None):
    """fp8q_gemm_rowscaled in the precise mode (FP16 MFMAs on the widened codes)."""
    M, N, K, out = _rowscaled_args("fp8q_gemm_rowscaled_precise", a_q, a_s, b_q, b_s, c)
    _invoke(lib.fp8q_gemm_rowscaled_precise, (_ptr(a_q), _ptr(a_s), _ptr(b_q), _ptr(b_s), M, N, K,
                                           _ptr(c), out, _stream(stream, a_q.device)), "fp8q_gemm_rowscaled_precise")


def _need(where, dev, *tensors):
    """_req of several (name, tensor, dtype, shape) on one device.  Nothing is
    looked up while all is right: calls that serve single tokens take about as
    long as their checks."""
    for name, t, dt, shape in tensors:
        try:
            if t.dtype is dt and t.shape == shape and t.device == dev and t.is_contiguous():
                continue
        except AttributeError:
            pass
        _req(where, name, t, [next(k for k in _DTYPES if _dt(k) is dt)], shape, dev)


def _act(where, act):
    if act not in _ACTS:
        raise ValueError(f"{where}: act = {act!r}, expected 'silu' or 'gelu_tanh'")
    return _ACTS[act]


def fp8q_quantize_token_i8(x, q, s, stream=None):
    """x: bf16 [M][K] -> q: int8 [M][Kp] (K up to a multiple of 16, zeros past
    K), s: float32 [M], one scale per row (in place)."""
    import torch
    wh = "fp8q_quantize_token_i8"
    M, K = _dims(wh, x, 2, "x")
    dev = x.device
    _need(wh, dev, ("x", x, torch.bfloat16, (M, K)), ("q", q, torch.int8, (M, -(-K // 16) * 16)),
          ("s", s, torch.float32, (M,)))
    _invoke(lib.fp8q_quantize_token_i8, (x.data_ptr(), M, K, q.data_ptr(), s.data_ptr(),
                                         _stream(stream, dev)), wh)


def _rows(where, a_q, w_q):
    """Rows of both operands, for the output's shape."""
    return _dims(where, a_q, 2, "a_q")[0], _dims(where, w_q, 2, "w_q")[0]


def _i8_args(where, a_q, a_s, w_q, w_s):
    import torch
    M, K = _dims(where, a_q, 2, "a_q")
    N, _ = _dims(where, w_q, 2, "w_q")
    if K % 16:
        raise ValueError(f"{where}: K = {K} is not a multiple of 16")
    dev = a_q.device
    _need(where, dev, ("a_q", a_q, torch.int8, (M, K)), ("a_s", a_s, torch.float32, (M,)),
          ("w_q", w_q, torch.int8, (N, K)), ("w_s", w_s, torch.float32, (N,)))
    return M, N, K, dev


def fp8q_gemm_i8(a_q, a_s, w_q, w_s, c, bias=None, stream=None):
    """c[M][N] (float32 or bfloat16) = (int8 a_q[M][K] x w_q[N][K]^T) * a_s[M]
    * w_s[N] (+ bias[N])."""
    wh = "fp8q_gemm_i8"
    M, N, K, dev = _i8_args(wh, a_q, a_s, w_q, w_s)
    _req(wh, "c", c, ["f32", "bf16"], (M, N), dev)
    if bias is not None:
        _req(wh, "bias", bias, ["f32"], (N,), dev)
    _invoke(lib.fp8q_gemm_i8, (a_q.data_ptr(), a_s.data_ptr(), w_q.data_ptr(), w_s.data_ptr(),
                               bias.data_ptr() if bias is not None else None, M, N, K,
                               c.data_ptr(), _out_code(wh, c), _stream(stream, dev)), wh)


def _gate_rows(where, N, multiple):
    if N % (2 * multiple):
        raise ValueError(f"{where}: w_q has {N} rows, expected gate and up rows"
                         + (f" in multiples of {multiple} each" if multiple > 1 else ""))


def fp8q_gemm_i8_gated(a_q, a_s, w_q, w_s, h, act="silu", stream=None):
    """h[M][F] = act(Y[:, :F]) * Y[:, F:], Y the int8 product of a_q[M][K] with
    the stacked gate and up weights w_q[2F][K], scaled by a_s[M] and w_s[2F]."""
    wh = "fp8q_gemm_i8_gated"
    M, N, K, dev = _i8_args(wh, a_q, a_s, w_q, w_s)
    _gate_rows(wh, N, 1)
    _req(wh, "h", h, ["f32", "bf16"], (M, N // 2), dev)
    _invoke(lib.fp8q_gemm_i8_gated, (a_q.data_ptr(), a_s.data_ptr(), w_q.data_ptr(),
                                     w_s.data_ptr(), M, N // 2, K, _act(wh, act), h.data_ptr(),
                                     _out_code(wh, h), _stream(stream, dev)), wh)


def _gated_args(where, a_q, a_s, off, w_q, w_s, h, gate_up):
    import torch
    M, K = _dims(where, a_q, 2, "a_q")
    lead = ()
    if off is not None:
        lead = (_dims(where, w_q, 3, "w_q")[0],)
    N = _dims(where, w_q, 2 + len(lead), "w_q")[-2]
    _mult128(where, K=K)
    _gate_rows(where, N, GROUP)
    dev = a_q.device
    _need(where, dev, ("a_q", a_q, torch.uint8, (M, K)),
          ("a_s", a_s, torch.float32, (K // GROUP, M)), ("w_q", w_q, torch.uint8, lead + (N, K)),
          ("w_s", w_s, torch.float32, lead + (N // GROUP, K // GROUP)))
    if off is not None:
        _need(where, dev, ("off", off, torch.int32, (lead[0] + 1,)))
    _req(where, "h", h, ["f32", "bf16"], (M, N // 2), dev)
    if gate_up is not None:
        _need(where, dev, ("gate_up", gate_up, torch.bfloat16, (M, N)))
    return M, N // 2, K, _out_code(where, h), dev


def fp8q_gemm_gated(a_q, a_s, w_q, w_s, h, act="silu", gate_up=None, stream=None):
    """h[M][F] = act(Y[:, :F]) * Y[:, F:], Y the block-scaled product of a_q
    with the stacked gate and up weights w_q[2F][K]; gate_up (bf16 [M][2F], or
    None) takes Y for the backward pass."""
    wh = "fp8q_gemm_gated"
    M, F, K, out, dev = _gated_args(wh, a_q, a_s, None, w_q, w_s, h, gate_up)
    _invoke(lib.fp8q_gemm_gated, (a_q.data_ptr(), a_s.data_ptr(), w_q.data_ptr(), w_s.data_ptr(),
                                  M, F, K, _act(wh, act), h.data_ptr(), out,
                                  gate_up.data_ptr() if gate_up is not None else None,
                                  _stream(stream, dev)), wh)


def fp8q_grouped_gemm_gated(a_q, a_s, off, w_q, w_s, h, act="silu", gate_up=None, stream=None):
    """fp8q_gemm_gated for routed experts: rows [off[e], off[e+1]) use expert
    e's w_q[e][2F][K]; off is a device int32[G+1]."""
    wh = "fp8q_grouped_gemm_gated"
    _dims(wh, off, 1, "off")
    M, F, K, out, dev = _gated_args(wh, a_q, a_s, off, w_q, w_s, h, gate_up)
    _invoke(lib.fp8q_grouped_gemm_gated, (a_q.data_ptr(), a_s.data_ptr(), M, off.data_ptr(),
                                          w_q.shape[0], w_q.data_ptr(), w_s.data_ptr(), F, K,
                                          _act(wh, act), h.data_ptr(), out,
                                          gate_up.data_ptr() if gate_up is not None else None,
                                          _stream(stream, dev)), wh)


def fp8q_gated_backward(dh, gate_up, q, s, qt, st, act="silu", mode="f32", stream=None):
    """dY = [dh * up * act'(gate) | dh * act(gate)] of dh: bf16 [M][F] and
    gate_up: bf16 [M][2F], quantized along the features (q: uint8 [M][2F], s:
    float32 [2F/128][M]) and along the tokens (qt: uint8 [2F][Mp], st: float32
    [Mp/128][2F], Mp = M up to a multiple of 128).  Either pair may be None."""
    import torch
    wh = "fp8q_gated_backward"
    M, F = _dims(wh, dh, 2, "dh")
    _mult128(wh, F=F)
    dev = dh.device
    _need(wh, dev, ("dh", dh, torch.bfloat16, (M, F)),
          ("gate_up", gate_up, torch.bfloat16, (M, 2 * F)))
    if (q is None) != (s is None) or (qt is None) != (st is None) or (q is None and qt is None):
        raise ValueError(f"{wh}: codes and scales come in pairs, and one pair at least")
    if q is not None:
        _need(wh, dev, ("q", q, torch.uint8, (M, 2 * F)),
              ("s", s, torch.float32, (2 * F // GROUP, M)))
    if qt is not None:
        groups = -(-M // GROUP)
        _need(wh, dev, ("qt", qt, torch.uint8, (2 * F, groups * GROUP)),
              ("st", st, torch.float32, (groups, 2 * F)))
    _invoke(lib.fp8q_gated_backward, (dh.data_ptr(), gate_up.data_ptr(), M, F, _act(wh, act),
                                      _MODES[mode], *(t.data_ptr() if t is not None else None
                                                      for t in (q, s, qt, st)),
                                      _stream(stream, dev)), wh)


def _positive_rows(where, N):
    if not 1 <= N <= 16384:
        raise ValueError(f"{where}: rows of {N} elements, expected 1 to 16384")


def _type_code(where, name, t):
    import torch
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{where}: {name} must be a torch.Tensor")
    code = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}.get(t.dtype)
    if code is None:
        raise ValueError(f"{where}: {name} has dtype {t.dtype}, expected float32 or bfloat16")
    return code


def fp8q_layer_norm(x, weight, bias, mean, rstd, y=None, q=None, s=None, eps=1e-5, mode="f32",
                    stream=None):
    """y = (x - mean) * rstd * weight (+ bias) of the rows of x (float32 or
    bfloat16 [M][N]; weight and bias float32 [N], bias may be None), into y
    (float32 or bfloat16 [M][N]), into q (uint8 [M][N]) and s (float32
    [N/128][M]) as E4M3, or into both; mean and rstd (float32 [M]) are written."""
    import torch
    wh = "fp8q_layer_norm"
    M, N = _dims(wh, x, 2, "x")
    _positive_rows(wh, N)
    dev = x.device
    xt = _type_code(wh, "x", x)
    _need(wh, dev, ("x", x, x.dtype, (M, N)), ("weight", weight, torch.float32, (N,)),
          ("mean", mean, torch.float32, (M,)), ("rstd", rstd, torch.float32, (M,)))
    if bias is not None:
        _need(wh, dev, ("bias", bias, torch.float32, (N,)))
    if (q is None) != (s is None) or (q is None and y is None):
        raise ValueError(f"{wh}: codes and scales come in a pair, and y or they are wanted")
    yt = OUT_F32
    if y is not None:
        _req(wh, "y", y, ["f32", "bf16"], (M, N), dev)
        yt = _type_code(wh, "y", y)
    if q is not None:
        _mult128(wh, N=N)
        _need(wh, dev, ("q", q, torch.uint8, (M, N)), ("s", s, torch.float32, (N // GROUP, M)))
    _invoke(lib.fp8q_layer_norm, (x.data_ptr(), xt, weight.data_ptr(), _at(bias), M, N, eps, _at(y),
                                  yt, _at(q), _at(s), _MODES[mode], mean.data_ptr(),
                                  rstd.data_ptr(), _stream(stream, dev)), wh)


def _at(t):
    return t.data_ptr() if t is not None else None


def layer_norm_backward_workspace(M, N):
    """Bytes of workspace that fp8q_layer_norm_backward takes."""
    return lib.fp8q_layer_norm_backward_workspace(M, N)


def fp8q_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, stream=None):
    """dx (of x's type) and the sums over all rows dweight and dbias (float32
    [N]; dbias may be None) from dy (float32 or bfloat16 [M][N]) and what
    fp8q_layer_norm read and wrote; workspace: uint8
    [layer_norm_backward_workspace(M, N)]."""
    import torch
    wh = "fp8q_layer_norm_backward"
    M, N = _dims(wh, x, 2, "x")
    _positive_rows(wh, N)
    dev = x.device
    xt = _type_code(wh, "x", x)
    _req(wh, "dy", dy, ["f32", "bf16"], (M, N), dev)
    _need(wh, dev, ("x", x, x.dtype, (M, N)), ("weight", weight, torch.float32, (N,)),
          ("mean", mean, torch.float32, (M,)), ("rstd", rstd, torch.float32, (M,)),
          ("dx", dx, x.dtype, (M, N)), ("dweight", dweight, torch.float32, (N,)),
          ("workspace", workspace, torch.uint8, (layer_norm_backward_workspace(M, N),)))
    if dbias is not None:
        _need(wh, dev, ("dbias", dbias, torch.float32, (N,)))
    _invoke(lib.fp8q_layer_norm_backward,
            (dy.data_ptr(), _type_code(wh, "dy", dy), x.data_ptr(), xt, weight.data_ptr(),
             mean.data_ptr(), rstd.data_ptr(), M, N, dx.data_ptr(), dweight.data_ptr(), _at(dbias),
             workspace.data_ptr(), _stream(stream, dev)), wh)


def expert_columns(M_total, G):
    """Columns of an operand whose M_total tokens are grouped by G experts, in
    groups of 128 that hold one expert's tokens each."""
    return lib.fp8q_expert_columns(M_total, G)


def _offsets(where, off, dev):
    import torch
    (n,) = _dims(where, off, 1, "off")
    if n < 2:
        raise ValueError(f"{where}: off has {n} elements, expected G + 1 of 1 expert at least")
    _need(where, dev, ("off", off, torch.int32, (n,)))
    return n - 1


def fp8q_grouped_quantize_act_t(x, off, q_t, s_t, mode="f32", stream=None):
    """x: bf16 [M_total][K], rows [off[e], off[e+1]) of expert e -> q_t: uint8
    [K][T], s_t: float32 [T/128][K], T = expert_columns(M_total, G) (in place)."""
    import torch
    wh = "fp8q_grouped_quantize_act_t"
    M, K = _dims(wh, x, 2, "x")
    _mult128(wh, K=K)
    dev = x.device
    G = _offsets(wh, off, dev)
    T = expert_columns(M, G)
    _need(wh, dev, ("x", x, torch.bfloat16, (M, K)), ("q_t", q_t, torch.uint8, (K, T)),
          ("s_t", s_t, torch.float32, (T // GROUP, K)))
    _invoke(lib.fp8q_grouped_quantize_act_t,
            (x.data_ptr(), M, off.data_ptr(), G, K, q_t.data_ptr(), s_t.data_ptr(), _MODES[mode],
             _stream(stream, dev)), wh)


def fp8q_grouped_gated_backward(dh, gate_up, off, q, s, qt, st, act="silu", mode="f32",
                                stream=None):
    """fp8q_gated_backward for routed experts: the groups of tokens of qt (uint8
    [2F][T]) and st (float32 [T/128][2F]) hold one expert's tokens each, T =
    expert_columns(M_total, G); rows of q and s past off[G] are not written."""
    import torch
    wh = "fp8q_grouped_gated_backward"
    M, F = _dims(wh, dh, 2, "dh")
    _mult128(wh, F=F)
    dev = dh.device
    G = _offsets(wh, off, dev)
    _need(wh, dev, ("dh", dh, torch.bfloat16, (M, F)),
          ("gate_up", gate_up, torch.bfloat16, (M, 2 * F)))
    if (q is None) != (s is None) or (qt is None) != (st is None) or (q is None and qt is None):
        raise ValueError(f"{wh}: codes and scales come in pairs, and one pair at least")
    if q is not None:
        _need(wh, dev, ("q", q, torch.uint8, (M, 2 * F)),
              ("s", s, torch.float32, (2 * F // GROUP, M)))
    if qt is not None:
        T = expert_columns(M, G)
        _need(wh, dev, ("qt", qt, torch.uint8, (2 * F, T)),
              ("st", st, torch.float32, (T // GROUP, 2 * F)))
    _invoke(lib.fp8q_grouped_gated_backward,
            (dh.data_ptr(), gate_up.data_ptr(), M, off.data_ptr(), G, F, _act(wh, act),
             _MODES[mode], _at(q), _at(s), _at(qt), _at(st), _stream(stream, dev)), wh)


def _grouped_rowscaled(wh, cfunc, a_q, a_s, b_q, b_s, off, c, stream):
    import torch
    N, T = _dims(wh, a_q, 2, "a_q")
    K, _ = _dims(wh, b_q, 2, "b_q")
    _mult128(wh, N=N, K=K, T=T)
    dev = a_q.device
    G = _offsets(wh, off, dev)
    _need(wh, dev, ("a_q", a_q, torch.uint8, (N, T)), ("a_s", a_s, torch.float32, (T // GROUP, N)),
          ("b_q", b_q, torch.uint8, (K, T)), ("b_s", b_s, torch.float32, (T // GROUP, K)))
    _req(wh, "c", c, ["f32", "bf16"], (G, N, K), dev)
    _invoke(cfunc, (a_q.data_ptr(), a_s.data_ptr(), b_q.data_ptr(), b_s.data_ptr(), T,
                    off.data_ptr(), G, N, K, c.data_ptr(), _out_code(wh, c),
                    _stream(stream, dev)), wh)


def fp8q_grouped_gemm_rowscaled(a_q, a_s, b_q, b_s, off, c, stream=None):
    """c[G][N][K] (float32 or bfloat16): of each expert its a_q [N][T] x b_q [K][T]^T
    over its groups of tokens, 1x128 row-group scales on both (the weight
    gradients dY^T X); off: the device int32[G+1] that grouped the tokens."""
    _grouped_rowscaled("fp8q_grouped_gemm_rowscaled", lib.fp8q_grouped_gemm_rowscaled, a_q, a_s,
                       b_q, b_s, off, c, stream)


def fp8q_grouped_gemm_rowscaled_precise(a_q, a_s, b_q, b_s, off, c, stream=None):
    """fp8q_grouped_gemm_rowscaled in the precise mode (FP16 MFMAs on the widened codes)."""
    _grouped_rowscaled("fp8q_grouped_gemm_rowscaled_precise",
                       lib.fp8q_grouped_gemm_rowscaled_precise, a_q, a_s, b_q, b_s, off, c, stream)


def _scalar(where, name, t, dtype, dev):
    import torch
    if not isinstance(t, torch.Tensor) or t.numel() != 1:
        raise ValueError(f"{where}: {name} must be a torch.Tensor of one element")
    _need(where, dev, (name, t, dtype, tuple(t.shape)))
    return t.data_ptr()


def _adamw_args(where, step, lr, betas, eps, weight_decay, grad_scale, dev):
    import torch
    a = AdamwArgs()
    if isinstance(lr, torch.Tensor):
        a.lr_dev = _scalar(where, "lr", lr, torch.float32, dev)
    else:
        a.lr = lr
    if isinstance(step, torch.Tensor):
        a.step_dev = _scalar(where, "step", step, torch.int32, dev)
    else:
        a.step = step
    if grad_scale is not None:
        a.grad_scale = _scalar(where, "grad_scale", grad_scale, torch.float32, dev)
    a.beta1, a.beta2 = betas
    a.eps, a.weight_decay = eps, weight_decay
    values = [(n, getattr(a, n)) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")]
    for n, v in values:
        if not 0 <= v < (1 if n.startswith("beta") else float("inf")):
            raise ValueError(f"{where}: {n} = {v}")
    if a.eps and not 2.0 ** -126 <= a.eps <= 2.0 ** 125:
        raise ValueError(f"{where}: eps = {a.eps}, expected 0 or 2^-126 to 2^125")
    if not a.step_dev and a.step < 1:
        raise ValueError(f"{where}: step = {step}, the first is 1")
    return a


def _adamw_call(where, params, grads, m, m_s, v, v_s, step, lr, betas, eps, weight_decay,
                grad_scale, copies, stream):
    import torch
    n = len(params)
    lists = {"grads": grads, "exp_avgs": m, "exp_avg_sqs": v, "exp_avg_scales": m_s,
             "exp_avg_sq_scales": v_s, "copies": copies}
    for name, l in lists.items():
        if l is not None and len(l) != n:
            raise ValueError(f"{where}: {n} params, {len(l)} {name}")
    if n == 0:
        return
    if not isinstance(params[0], torch.Tensor):
        raise ValueError(f"{where}: params must be torch.Tensors")
    dev = params[0].device
    eight = m_s is not None
    grad_type = _type_code(where, "grads[0]", grads[0])
    moment = torch.uint8 if eight else torch.float32
    array = (AdamwTensor * n)()
    for i, (p, a) in enumerate(zip(params, array)):
        if not isinstance(p, torch.Tensor):
            raise ValueError(f"{where}: params[{i}] must be a torch.Tensor")
        shape, count = tuple(p.shape), p.numel()
        _need(where, dev, (f"params[{i}]", p, torch.float32, shape),
              (f"grads[{i}]", grads[i], grads[0].dtype, shape),
              (f"exp_avgs[{i}]", m[i], moment, shape), (f"exp_avg_sqs[{i}]", v[i], moment, shape))
        a.p, a.g, a.m, a.v, a.n = p.data_ptr(), grads[i].data_ptr(), m[i].data_ptr(), \
            v[i].data_ptr(), count
        if eight:
            groups = (-(-count // GROUP),)
            _need(where, dev, (f"exp_avg_scales[{i}]", m_s[i], torch.float32, groups),
                  (f"exp_avg_sq_scales[{i}]", v_s[i], torch.float32, groups))
            a.m_s, a.v_s = m_s[i].data_ptr(), v_s[i].data_ptr()
        if copies is not None:
            _need(where, dev, (f"copies[{i}]", copies[i], torch.bfloat16, shape))
            a.copy = copies[i].data_ptr()
    args = _adamw_args(where, step, lr, betas, eps, weight_decay, grad_scale, dev)
    _invoke(lib.fp8q_adamw, (array, n, args, grad_type, MOMENTS_E4M3 if eight else MOMENTS_F32,
                             _stream(stream, dev)), where,
            [t for l in (params, m, v, m_s, v_s, copies) if l is not None for t in l])


def fp8q_adamw(params, grads, exp_avgs, exp_avg_sqs, step, lr=1e-3, betas=(0.9, 0.95), eps=1e-8,
               weight_decay=0.1, exp_avg_scales=None, exp_avg_sq_scales=None, grad_scale=None,
               copies=None, stream=None):
    """One AdamW step over lists of tensors, in place: see adamw and adamw_8bit
    (which have the scales)."""
    if (exp_avg_scales is None) != (exp_avg_sq_scales is None):
        raise ValueError("fp8q_adamw: both moments have scales, or neither")
    _adamw_call("fp8q_adamw", params, grads, exp_avgs, exp_avg_scales, exp_avg_sqs,
                exp_avg_sq_scales, step, lr, betas, eps, weight_decay, grad_scale, copies, stream)


# ---------------------------------------------------------- allocation helpers
def _new(stream, device, *wanted):
    """Tensors of the (shape, dtype) pairs, None for a None, that a call on `stream`
    (None: the current one) writes.

    torch hands a freed block out again to the stream it was allocated on, whose order
    keeps the old use before the new.  So a named stream's tensors are allocated on
    that stream: a block of the current one's may be in use by work of its that is
    still pending.  The caller goes on with them on the current stream: it is recorded,
    and a block that is dropped waits for what the current stream does with it."""
    import torch

    def made():
        return [w and torch.empty(w[0], dtype=w[1], device=device) for w in wanted]
    if stream is None or device.type != "cuda":
        return made()
    here = torch.cuda.current_stream(device)
    if stream.cuda_stream == here.cuda_stream:
        return made()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        tensors = made()
    for t in tensors:
        if t is not None:
            t.record_stream(here)
    return tensors


def quantize_act(x, mode="f32", stream=None):
    import torch
    M, K = x.shape
    q, s = _new(stream, x.device, ((M, K), torch.uint8), ((K // GROUP, M), torch.float32))
    fp8q_quantize_act(x, q, s, mode, stream)
    return q, s


def quantize_weight(w, mode="f32", stream=None):
    import torch
    N, K = w.shape
    q, s = _new(stream, w.device, ((N, K), torch.uint8), ((N // GROUP, K // GROUP), torch.float32))
    fp8q_quantize_weight(w, q, s, mode, stream)
    return q, s


def quantize_act_t(x, mode="f32", stream=None):
    import torch
    M, K = x.shape
    q, s = _new(stream, x.device, ((K, M), torch.uint8), ((M // GROUP, K), torch.float32))
    fp8q_quantize_act_t(x, q, s, mode, stream)
    return q, s


def quantize_weight_t(w, mode="f32", stream=None):
    import torch
    N, K = w.shape
    q, s = _new(stream, w.device, ((K, N), torch.uint8), ((K // GROUP, N // GROUP), torch.float32))
    fp8q_quantize_weight_t(w, q, s, mode, stream)
    return q, s


def gemm_rowscaled(a_q, a_s, b_q, b_s, out_dtype=None, stream=None, precise=False):
    import torch
    out_dtype = out_dtype or torch.float32
    (c,) = _new(stream, a_q.device, ((a_q.shape[0], b_q.shape[0]), out_dtype))
    f = fp8q_gemm_rowscaled_precise if precise else fp8q_gemm_rowscaled
    f(a_q, a_s, b_q, b_s, c, stream)
    return c


def gemm(a_q, a_s, w_q, w_s, out_dtype=None, stream=None, precise=False, mfma_scaled=False):
    import torch
    out_dtype = out_dtype or torch.float32
    (c,) = _new(stream, a_q.device, ((a_q.shape[0], w_q.shape[0]), out_dtype))
    assert not (precise and mfma_scaled), "one GEMM mode"
    f = fp8q_gemm_precise if precise else fp8q_gemm_mfma_scaled if mfma_scaled else fp8q_gemm
    f(a_q, a_s, w_q, w_s, c, stream)
    return c


def gemm_fused(x, w_q, w_s, mode="f32", out_dtype=None, stream=None):
    import torch
    out_dtype = out_dtype or torch.float32
    (c,) = _new(stream, x.device, ((x.shape[0], w_q.shape[0]), out_dtype))
    fp8q_gemm_fused(x, w_q, w_s, c, mode, stream)
    return c


def grouped_gemm_fused(x, off, w_q, w_s, mode="f32", out_dtype=None, stream=None):
    import torch
    out_dtype = out_dtype or torch.float32
    (c,) = _new(stream, x.device, ((x.shape[0], w_q.shape[1]), out_dtype))
    fp8q_grouped_gemm_fused(x, off, w_q, w_s, c, mode, stream)
    return c


def grouped_gemm(a_q, a_s, off, w_q, w_s, out_dtype=None, stream=None, precise=False):
    import torch
    out_dtype = out_dtype or torch.float32
    (c,) = _new(stream, a_q.device, ((a_q.shape[0], w_q.shape[1]), out_dtype))
    f = fp8q_grouped_gemm_precise if precise else fp8q_grouped_gemm
    f(a_q, a_s, off, w_q, w_s, c, stream)
    return c


_native = None


class _PythonPath:
    """In the compiled module's place: takes no call, so each goes the Python path."""

    @staticmethod
    def _decline(*args):
        return None

    quantize_token_i8 = gemm_i8 = gemm_i8_gated = gemm_gated = gated_backward = _decline
    layer_norm = layer_norm_backward = grouped_quantize_act_t = _decline
    grouped_gated_backward = grouped_gemm_rowscaled = adamw = _decline


def _compiled():
    """The module of csrc/calls.cpp with this library's entry points (or, where it
    cannot be loaded, _PythonPath), and the output codes of the dtypes it
    allocates."""
    global _native, _OUT_OF
    import torch       # its libraries first
    _OUT_OF = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}
    try:
        from . import _calls
    except ImportError as e:   # not built, or against another torch
        warnings.warn(f"the compiled calls cannot be loaded ({e}); the feed-forward helpers "
                      "take their Python path, about 10 us a call slower", RuntimeWarning,
                      stacklevel=3)
        _native = _PythonPath
        return _native
    _calls.entries(*(ctypes.cast(getattr(lib, "fp8q_" + n), _p).value for n in
                     ("quantize_token_i8", "gemm_i8", "gemm_i8_gated", "gemm_gated",
                      "grouped_gemm_gated", "gated_backward", "layer_norm",
                      "layer_norm_backward_workspace", "layer_norm_backward", "expert_columns",
                      "grouped_quantize_act_t", "grouped_gated_backward",
                      "grouped_gemm_rowscaled", "grouped_gemm_rowscaled_precise", "adamw")))
    _native = _calls
    return _native


def _refused(status, where):
    raise Fp8qError(status, where)


def quantize_token_i8(x, stream=None):
    """x: bf16 [M][K] -> (int8 codes [M][Kp], float32 scales [M]); Kp is K up to
    a multiple of 16, with zero codes past K."""
    wh = "fp8q_quantize_token_i8"
    if stream is None:
        r = (_native or _compiled()).quantize_token_i8(x)
        if r is not None:
            return r if type(r) is not int else _refused(r, wh)
    import torch
    M, K = _dims(wh, x, 2, "x")
    q, s = _new(stream, x.device, ((M, -(-K // 16) * 16), torch.int8), ((M,), torch.float32))
    fp8q_quantize_token_i8(x, q, s, stream)
    return q, s


def gemm_i8(a_q, a_s, w_q, w_s, bias=None, out_dtype=None, stream=None):
    wh = "fp8q_gemm_i8"
    if stream is None:
        native = _native or _compiled()
        out = OUT_F32 if out_dtype is None else _OUT_OF.get(out_dtype)
        if out is not None:
            r = native.gemm_i8(a_q, a_s, w_q, w_s, bias, out)
            if r is not None:
                return r if type(r) is not int else _refused(r, wh)
    import torch
    M, N = _rows(wh, a_q, w_q)
    (c,) = _new(stream, a_q.device, ((M, N), out_dtype or torch.float32))
    fp8q_gemm_i8(a_q, a_s, w_q, w_s, c, bias, stream)
    return c


def gemm_i8_gated(a_q, a_s, w_q, w_s, act="silu", out_dtype=None, stream=None):
    """h = act(gate) * up (bfloat16 unless out_dtype says float32)."""
    wh = "fp8q_gemm_i8_gated"
    if stream is None:
        native = _native or _compiled()
        out = OUT_BF16 if out_dtype is None else _OUT_OF.get(out_dtype)
        if out is not None:
            r = native.gemm_i8_gated(a_q, a_s, w_q, w_s, _act(wh, act), out)
            if r is not None:
                return r if type(r) is not int else _refused(r, wh)
    import torch
    M, N = _rows(wh, a_q, w_q)
    (h,) = _new(stream, a_q.device, ((M, N // 2), out_dtype or torch.bfloat16))
    fp8q_gemm_i8_gated(a_q, a_s, w_q, w_s, h, act, stream)
    return h


def _gated(wh, a_q, a_s, off, w_q, w_s, act, out_dtype, save_gate_up, stream):
    if stream is None:
        native = _native or _compiled()
        out = OUT_BF16 if out_dtype is None else _OUT_OF.get(out_dtype)
        if out is not None:
            r = native.gemm_gated(a_q, a_s, off, w_q, w_s, _act(wh, act), out, save_gate_up)
            if r is not None:
                return r if type(r) is not int else _refused(r, wh)
    import torch
    M = _dims(wh, a_q, 2, "a_q")[0]
    N = _dims(wh, w_q, 2 if off is None else 3, "w_q")[-2]
    h, gu = _new(stream, a_q.device, ((M, N // 2), out_dtype or torch.bfloat16),
                 ((M, N), torch.bfloat16) if save_gate_up else None)
    if off is None:
        fp8q_gemm_gated(a_q, a_s, w_q, w_s, h, act, gu, stream)
    else:
        fp8q_grouped_gemm_gated(a_q, a_s, off, w_q, w_s, h, act, gu, stream)
    return (h, gu) if save_gate_up else h


def gemm_gated(a_q, a_s, w_q, w_s, act="silu", out_dtype=None, save_gate_up=False, stream=None):
    """h = act(gate) * up (bfloat16 unless out_dtype says float32); with
    save_gate_up, (h, the bfloat16 [gate | up] the backward pass takes)."""
    return _gated("fp8q_gemm_gated", a_q, a_s, None, w_q, w_s, act, out_dtype, save_gate_up, stream)


def grouped_gemm_gated(a_q, a_s, off, w_q, w_s, act="silu", out_dtype=None, save_gate_up=False,
                       stream=None):
    """gemm_gated by expert; rows at or past off[G] are not written."""
    wh = "fp8q_grouped_gemm_gated"
    _dims(wh, off, 1, "off")
    return _gated(wh, a_q, a_s, off, w_q, w_s, act, out_dtype, save_gate_up, stream)


def _both_forms(stream, device, M, F, groups, rows, tokens):
    """q, s, qt, st of the gated block's backward pass, of M rows and `groups` of tokens."""
    import torch
    return _new(stream, device, ((M, 2 * F), torch.uint8) if rows else None,
                ((2 * F // GROUP, M), torch.float32) if rows else None,
                ((2 * F, groups * GROUP), torch.uint8) if tokens else None,
                ((groups, 2 * F), torch.float32) if tokens else None)


def gated_backward(dh, gate_up, act="silu", mode="f32", rows=True, tokens=True, stream=None):
    """(q, s, qt, st): dY in E4M3 along the features and along the tokens, for
    gemm (dX = dY W) and gemm_rowscaled (dW = dY^T X).  rows=False or
    tokens=False leaves that pair out (None)."""
    wh = "fp8q_gated_backward"
    if stream is None:
        r = (_native or _compiled()).gated_backward(dh, gate_up, _act(wh, act), _MODES[mode], rows,
                                                    tokens)
        if r is not None:
            return r if type(r) is not int else _refused(r, wh)
    M, F = _dims(wh, dh, 2, "dh")
    q, s, qt, st = _both_forms(stream, dh.device, M, F, -(-M // GROUP), rows, tokens)
    fp8q_gated_backward(dh, gate_up, q, s, qt, st, act, mode, stream)
    return q, s, qt, st


def _norm(x, weight, bias, eps, y_dtype, codes, mode, stream):
    """The Python path of both calls below."""
    import torch
    wh = "fp8q_layer_norm"
    M, N = _dims(wh, x, 2, "x")
    _positive_rows(wh, N)
    if codes:
        _mult128(wh, N=N)
    y, q, s, mean, rstd = _new(
        stream, x.device, ((M, N), y_dtype) if y_dtype is not None else None,
        ((M, N), torch.uint8) if codes else None, ((N // GROUP, M), torch.float32) if codes else None,
        ((M,), torch.float32), ((M,), torch.float32))
    fp8q_layer_norm(x, weight, bias, mean, rstd, y, q, s, eps, mode, stream)
    return y, q, s, mean, rstd


def layer_norm(x, weight, bias=None, eps=1e-5, out_dtype=None, stream=None):
    """(y, mean, rstd): layer norm of the rows of x (float32 or bfloat16 [M][N],
    weight and bias float32 [N]); y is bfloat16 unless out_dtype says float32."""
    if stream is None:
        native = _native or _compiled()
        out = OUT_BF16 if out_dtype is None else _OUT_OF.get(out_dtype)
        if out is not None:
            r = native.layer_norm(x, weight, bias, eps, out, False, SCALE_F32)
            if r is not None:
                return r if type(r) is not int else _refused(r, "fp8q_layer_norm")
    import torch
    y, _, _, mean, rstd = _norm(x, weight, bias, eps, out_dtype or torch.bfloat16, False, "f32",
                                stream)
    return y, mean, rstd


def layer_norm_quantized(x, weight, bias=None, eps=1e-5, mode="f32", save_y=False, out_dtype=None,
                         stream=None):
    """(q, s, mean, rstd): layer norm written as the E4M3 operand of gemm, from y
    in float32; with save_y, (q, s, mean, rstd, y), y as layer_norm's."""
    if stream is None:
        native = _native or _compiled()
        out = -1 if not save_y else OUT_BF16 if out_dtype is None else _OUT_OF.get(out_dtype)
        if out is not None:
            r = native.layer_norm(x, weight, bias, eps, out, True, _MODES[mode])
            if r is not None:
                return r if type(r) is not int else _refused(r, "fp8q_layer_norm")
    import torch
    y, q, s, mean, rstd = _norm(x, weight, bias, eps,
                                (out_dtype or torch.bfloat16) if save_y else None, True, mode,
                                stream)
    return (q, s, mean, rstd, y) if save_y else (q, s, mean, rstd)


def layer_norm_backward(dy, x, weight, mean, rstd, bias=True, stream=None):
    """(dx, dweight, dbias): the gradients of layer_norm, dx of x's type, the
    others float32; bias=False leaves dbias out (None)."""
    wh = "fp8q_layer_norm_backward"
    if stream is None:
        r = (_native or _compiled()).layer_norm_backward(dy, x, weight, mean, rstd, bias)
        if r is not None:
            return r if type(r) is not int else _refused(r, wh)
    import torch
    M, N = _dims(wh, x, 2, "x")
    dx, dweight, dbias, work = _new(
        stream, x.device, ((M, N), x.dtype), ((N,), torch.float32),
        ((N,), torch.float32) if bias else None, ((layer_norm_backward_workspace(M, N),), torch.uint8))
    fp8q_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, work, stream)
    return dx, dweight, dbias


def grouped_quantize_act_t(x, off, mode="f32", stream=None):
    """(q_t, s_t): x (bf16 [M_total][K], rows grouped by expert) in E4M3 along the
    tokens, for grouped_gemm_rowscaled: uint8 [K][T] and float32 [T/128][K], T =
    expert_columns(M_total, G)."""
    wh = "fp8q_grouped_quantize_act_t"
    if stream is None:
        r = (_native or _compiled()).grouped_quantize_act_t(x, off, _MODES[mode])
        if r is not None:
            return r if type(r) is not int else _refused(r, wh)
    import torch
    M, K = _dims(wh, x, 2, "x")
    T = expert_columns(M, _offsets(wh, off, x.device))
    q, s = _new(stream, x.device, ((K, T), torch.uint8), ((T // GROUP, K), torch.float32))
    fp8q_grouped_quantize_act_t(x, off, q, s, mode, stream)
    return q, s


def grouped_gated_backward(dh, gate_up, off, act="silu", mode="f32", rows=True, tokens=True,
                           stream=None):
    """(q, s, qt, st): gated_backward by expert, for grouped_gemm (dX) and
    grouped_gemm_rowscaled (dW); rows of q and s past off[G] are not written."""
    wh = "fp8q_grouped_gated_backward"
    if stream is None:
        r = (_native or _compiled()).grouped_gated_backward(dh, gate_up, off, _act(wh, act),
                                                            _MODES[mode], rows, tokens)
        if r is not None:
            return r if type(r) is not int else _refused(r, wh)
    M, F = _dims(wh, dh, 2, "dh")
    groups = expert_columns(M, _offsets(wh, off, dh.device)) // GROUP
    q, s, qt, st = _both_forms(stream, dh.device, M, F, groups, rows, tokens)
    fp8q_grouped_gated_backward(dh, gate_up, off, q, s, qt, st, act, mode, stream)
    return q, s, qt, st


def grouped_gemm_rowscaled(a_q, a_s, b_q, b_s, off, out_dtype=None, stream=None, precise=False):
    """[G][N][K]: the weight gradients of all experts from both operands' codes
    along the tokens (grouped_quantize_act_t, grouped_gated_backward); zeros for
    an expert without tokens."""
    wh = "fp8q_grouped_gemm_rowscaled" + ("_precise" if precise else "")
    if stream is None:
        native = _native or _compiled()
        out = OUT_F32 if out_dtype is None else _OUT_OF.get(out_dtype)
        if out is not None:
            r = native.grouped_gemm_rowscaled(a_q, a_s, b_q, b_s, off, out, precise)
            if r is not None:
                return r if type(r) is not int else _refused(r, wh)
    import torch
    N, K = _rows(wh, a_q, b_q)
    G = _offsets(wh, off, a_q.device)
    (c,) = _new(stream, a_q.device, ((G, N, K), out_dtype or torch.float32))
    f = fp8q_grouped_gemm_rowscaled_precise if precise else fp8q_grouped_gemm_rowscaled
    f(a_q, a_s, b_q, b_s, off, c, stream)
    return c


def _adamw(params, grads, m, m_s, v, v_s, step, lr, betas, eps, weight_decay, grad_scale, copies,
           stream):
    wh = "fp8q_adamw"
    if stream is None:
        r = (_native or _compiled()).adamw(params, grads, m, m_s, v, v_s, copies, step, lr, *betas,
                                           eps, weight_decay, grad_scale)
        if r is not None:
            return None if r == OK else _refused(r, wh)
    _adamw_call(wh, params, grads, m, m_s, v, v_s, step, lr, betas, eps, weight_decay, grad_scale,
                copies, stream)


def adamw(params, grads, exp_avgs, exp_avg_sqs, step, lr=1e-3, betas=(0.9, 0.95), eps=1e-8,
          weight_decay=0.1, grad_scale=None, copies=None, stream=None):
    """One AdamW step over lists of tensors, in place.  params (masters) and both
    moments are float32, grads float32 or bfloat16 (one type), each of its
    parameter's shape; copies, if given, take the new parameters as bfloat16.
    step counts from 1.  step and lr may be device tensors of one element (int32
    and float32), which a captured graph reads at each replay; grad_scale
    (float32, on the device) multiplies the gradients."""
    _adamw(params, grads, exp_avgs, None, exp_avg_sqs, None, step, lr, betas, eps, weight_decay,
           grad_scale, copies, stream)


def adamw_8bit(params, grads, exp_avgs, exp_avg_scales, exp_avg_sqs, exp_avg_sq_scales, step,
               lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, grad_scale=None,
               copies=None, stream=None):
    """adamw with both moments in E4M3: exp_avgs holds the codes (uint8, the
    parameter's shape) of the first moment, exp_avg_sqs those of the second
    moment's square root, 128 consecutive elements with one scale (float32
    [ceil(n/128)]).  Zero codes and scales are the state before the first step.
    The codes are rounded with a dither of the element's place and the step, so
    that a moment which moves by less than a code's step each time does not stay
    where it is.  An element whose gradient is not finite, or so large that its
    square overflows, is NaN from the next step on at the latest; the others of
    its group keep their moments."""
    _adamw(params, grads, exp_avgs, exp_avg_scales, exp_avg_sqs, exp_avg_sq_scales, step, lr,
           betas, eps, weight_decay, grad_scale, copies, stream)
