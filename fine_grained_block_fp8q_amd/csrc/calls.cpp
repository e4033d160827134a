// The allocating calls of the feed-forward operators, compiled.
//
// A product for one token takes the GPU 6 us; checked, allocated and launched
// from Python its call took 14.  These functions take 4.4 us with one output and
// 5.8 with four, of which the launch is 3.8 (outputs allocated through torch's
// dispatcher: 4.5 and 6.6).  They serve the calls where everything is right:
// every argument a tensor of the right type and shape, contiguous, on the
// current device; the outputs are allocated, the C entry point called on torch's
// current stream, and the outputs returned.  They return an int (the status)
// when the entry point refuses, and None when an argument is not as it should
// be: the Python function then takes its own path, whose checks raise.  They
// return None too while something is to see or fill torch's allocations (a
// dispatch mode, or the deterministic filling of uninitialized memory), which
// these do not show it.  (Function modes do not count: the default device is one,
// and the allocations name theirs.)
//
// Nothing is kept from one call for the next.

#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/Context.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <vector>

#include "fp8q.h"

namespace {

using at::Tensor;

// C entry points of the library that the package has loaded, in this order.
struct Entries {
  decltype(&fp8q_quantize_token_i8) quantize_token_i8;
  decltype(&fp8q_gemm_i8) gemm_i8;
  decltype(&fp8q_gemm_i8_gated) gemm_i8_gated;
  decltype(&fp8q_gemm_gated) gemm_gated;
  decltype(&fp8q_grouped_gemm_gated) grouped_gemm_gated;
  decltype(&fp8q_gated_backward) gated_backward;
  decltype(&fp8q_layer_norm) layer_norm;
  decltype(&fp8q_layer_norm_backward_workspace) layer_norm_backward_workspace;
  decltype(&fp8q_layer_norm_backward) layer_norm_backward;
  decltype(&fp8q_expert_columns) expert_columns;
  decltype(&fp8q_grouped_quantize_act_t) grouped_quantize_act_t;
  decltype(&fp8q_grouped_gated_backward) grouped_gated_backward;
  decltype(&fp8q_grouped_gemm_rowscaled) grouped_gemm_rowscaled;
  decltype(&fp8q_grouped_gemm_rowscaled_precise) grouped_gemm_rowscaled_precise;
  decltype(&fp8q_adamw) adamw;
} entries;
constexpr Py_ssize_t kEntries = sizeof(Entries) / sizeof(void*);

const Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool allocations_watched() {
  const auto& context = at::globalContext();
  return c10::impl::TorchDispatchModeTLS::any_modes_set() ||
         (context.deterministicAlgorithms() && context.deterministicFillUninitializedMemory());
}

// Tensors of one call: all on the device of the first, which is current.
struct Call {
  at::Device dev;
  bool ok;
  explicit Call(const Tensor& first)
      : dev(first.device()),
        ok(dev.is_cuda() && dev.index() == c10::hip::current_device() && !allocations_watched()) {}
  void need(const Tensor& t, at::ScalarType type, at::IntArrayRef sizes) {
    ok = ok && t.scalar_type() == type && t.device() == dev && t.sizes() == sizes &&
         t.is_contiguous();
  }
  Tensor make(at::ScalarType type, at::IntArrayRef sizes) const {
    return Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
  }
  hipStream_t stream() const { return c10::hip::getCurrentHIPStream(dev.index()).stream(); }
};

// The truth of a flag; false with Python's error set where it has none.
bool truth(PyObject* o, bool& value) {
  const int t = PyObject_IsTrue(o);
  value = t == 1;
  return t >= 0;
}

template <class T = void>
T* at_(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

PyObject* answer(fp8q_status st, const Tensor& a) {
  return st == FP8Q_OK ? THPVariable_Wrap(a) : PyLong_FromLong(st);
}

PyObject* wrap_or_none(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

template <class... Ts>
PyObject* answers(fp8q_status st, const Ts&... ts) {
  if (st != FP8Q_OK) return PyLong_FromLong(st);
  const Tensor* all[] = {&ts...};
  PyObject* r = PyTuple_New(sizeof...(ts));
  if (!r) return nullptr;
  for (size_t i = 0; i < sizeof...(ts); ++i) {
    PyObject* o = wrap_or_none(*all[i]);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

at::ScalarType out_type(int out) { return out == FP8Q_OUT_BF16 ? at::kBFloat16 : at::kFloat; }

// A function body: torch's errors (an allocation that fails) become Python's,
// as they do in torch's own functions.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

#define NEEDS(n)                                                                    \
  if (nargs != n) {                                                                 \
    PyErr_Format(PyExc_TypeError, "%s takes %d arguments, got %zd", __func__, n, nargs); \
    return nullptr;                                                                 \
  }

// quantize_token_i8(x)
PyObject* quantize_token_i8(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS(1)
  return guarded([&]() -> PyObject* {
    const Tensor* x = tensor(args[0]);
    if (!x || x->dim() != 2) Py_RETURN_NONE;
    const int64_t M = x->size(0), K = x->size(1);
    Call c(*x);
    c.need(*x, at::kBFloat16, {M, K});
    if (!c.ok) Py_RETURN_NONE;
    const Tensor q = c.make(at::kChar, {M, (K + 15) / 16 * 16}), s = c.make(at::kFloat, {M});
    return answers(entries.quantize_token_i8(at_(*x), M, K, at_<int8_t>(q), at_<float>(s),
                                             c.stream()),
                   q, s);
  });
}

// gemm_i8(a_q, a_s, w_q, w_s, bias or None, out)
PyObject* gemm_i8(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS(6)
  return guarded([&]() -> PyObject* {
    const Tensor *a = tensor(args[0]), *as = tensor(args[1]), *w = tensor(args[2]),
                 *ws = tensor(args[3]);
    const Tensor* bias = args[4] == Py_None ? nullptr : tensor(args[4]);
    if (!a || !as || !w || !ws || (args[4] != Py_None && !bias) || a->dim() != 2 || w->dim() != 2)
      Py_RETURN_NONE;
    const int64_t M = a->size(0), K = a->size(1), N = w->size(0);
    Call c(*a);
    c.need(*a, at::kChar, {M, K});
    c.need(*as, at::kFloat, {M});
    c.need(*w, at::kChar, {N, K});
    c.need(*ws, at::kFloat, {N});
    if (bias) c.need(*bias, at::kFloat, {N});
    if (!c.ok || K % 16) Py_RETURN_NONE;
    const int out = (int)PyLong_AsLong(args[5]);
    const Tensor y = c.make(out_type(out), {M, N});
    return answer(entries.gemm_i8(at_<int8_t>(*a), at_<float>(*as), at_<int8_t>(*w),
                                  at_<float>(*ws), bias ? at_<float>(*bias) : nullptr, M, N, K,
                                  at_(y), (fp8q_out_dtype)out, c.stream()),
                  y);
  });
}

// gemm_i8_gated(a_q, a_s, w_q, w_s, act, out)
PyObject* gemm_i8_gated(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS(6)
  return guarded([&]() -> PyObject* {
    const Tensor *a = tensor(args[0]), *as = tensor(args[1]), *w = tensor(args[2]),
                 *ws = tensor(args[3]);
    if (!a || !as || !w || !ws || a->dim() != 2 || w->dim() != 2) Py_RETURN_NONE;
    const int64_t M = a->size(0), K = a->size(1), N = w->size(0);
    Call c(*a);
    c.need(*a, at::kChar, {M, K});
    c.need(*as, at::kFloat, {M});
    c.need(*w, at::kChar, {N, K});
    c.need(*ws, at::kFloat, {N});
    if (!c.ok || K % 16 || N % 2) Py_RETURN_NONE;
    const int out = (int)PyLong_AsLong(args[5]);
    const Tensor h = c.make(out_type(out), {M, N / 2});
    return answer(entries.gemm_i8_gated(at_<int8_t>(*a), at_<float>(*as), at_<int8_t>(*w),
                                        at_<float>(*ws), M, N / 2, K,
                                        (fp8q_activation)PyLong_AsLong(args[4]), at_(h),
                                        (fp8q_out_dtype)out, c.stream()),
                  h);
  });
}

// gemm_gated(a_q, a_s, off or None, w_q, w_s, act, out, save): by expert with off
PyObject* gemm_gated(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS(8)
  return guarded([&]() -> PyObject* {
    const bool grouped = args[2] != Py_None;
    const Tensor *a = tensor(args[0]), *as = tensor(args[1]), *off = tensor(args[2]),
                 *w = tensor(args[3]), *ws = tensor(args[4]);
    if (!a || !as || !w || !ws || (grouped && !off) || a->dim() != 2 ||
        w->dim() != (grouped ? 3 : 2))
      Py_RETURN_NONE;
    const int64_t M = a->size(0), K = a->size(1), N = w->size(-2), G = grouped ? w->size(0) : 1;
    Call c(*a);
    c.need(*a, at::kByte, {M, K});
    c.need(*as, at::kFloat, {K / 128, M});
    if (grouped) {
      c.need(*off, at::kInt, {G + 1});
      c.need(*w, at::kByte, {G, N, K});
      c.need(*ws, at::kFloat, {G, N / 128, K / 128});
    } else {
      c.need(*w, at::kByte, {N, K});
      c.need(*ws, at::kFloat, {N / 128, K / 128});
    }
    if (!c.ok || K % 128 || N % 256 || G > INT32_MAX) Py_RETURN_NONE;
    const auto act = (fp8q_activation)PyLong_AsLong(args[5]);
    const int out = (int)PyLong_AsLong(args[6]);
    bool save;
    if (!truth(args[7], save)) return nullptr;
    const Tensor h = c.make(out_type(out), {M, N / 2});
    const Tensor gu = save ? c.make(at::kBFloat16, {M, N}) : Tensor();
    const fp8q_status st =
        grouped ? entries.grouped_gemm_gated(at_<uint8_t>(*a), at_<float>(*as), M, at_<int32_t>(*off),
                                             (int32_t)G, at_<uint8_t>(*w), at_<float>(*ws), N / 2, K,
                                             act, at_(h), (fp8q_out_dtype)out, at_(gu), c.stream())
                : entries.gemm_gated(at_<uint8_t>(*a), at_<float>(*as), at_<uint8_t>(*w),
                                     at_<float>(*ws), M, N / 2, K, act, at_(h), (fp8q_out_dtype)out,
                                     at_(gu), c.stream());
    return save ? answers(st, h, gu) : answer(st, h);
  });
}

// gated_backward(dh, gate_up, act, mode, rows, tokens)
PyObject* gated_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS(6)
  return guarded([&]() -> PyObject* {
    const Tensor *dh = tensor(args[0]), *gu = tensor(args[1]);
    if (!dh || !gu || dh->dim() != 2) Py_RETURN_NONE;
    const int64_t M = dh->size(0), F = dh->size(1), groups = (M + 127) / 128;
    Call c(*dh);
    c.need(*dh, at::kBFloat16, {M, F});
    c.need(*gu, at::kBFloat16, {M, 2 * F});
    bool rows, tokens;
    if (!truth(args[4], rows) || !truth(args[5], tokens)) return nullptr;
    if (!c.ok || F % 128 || !(rows || tokens)) Py_RETURN_NONE;
    Tensor q, s, qt, st;
    if (rows) {
      q = c.make(at::kByte, {M, 2 * F});
      s = c.make(at::kFloat, {2 * F / 128, M});
    }
    if (tokens) {
      qt = c.make(at::kByte, {2 * F, groups * 128});
      st = c.make(at::kFloat, {groups, 2 * F});
    }
    return answers(entries.gated_backward(at_(*dh), at_(*gu), M, F,
                                          (fp8q_activation)PyLong_AsLong(args[2]),
                                          (fp8q_scale_mode)PyLong_AsLong(args[3]), at_<uint8_t>(q),
                                          at_<float>(s), at_<uint8_t>(qt), at_<float>(st),
                                          c.stream()),
                   q, s, qt, st);
  });
}

bool real(at::ScalarType t) { return t == at::kFloat || t == at::kBFloat16; }
fp8q_out_dtype type_code(at::ScalarType t) {
  return t == at::kBFloat16 ? FP8Q_OUT_BF16 : FP8Q_OUT_F32;
}

// layer_norm(x, weight, bias or None, eps, y's type or -1, codes, mode): (y, mean,
// rstd), with codes (q, s, mean, rstd) and y behind them where it is wanted
PyObject* layer_norm(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS(7)
  return guarded([&]() -> PyObject* {
    const Tensor *x = tensor(args[0]), *w = tensor(args[1]);
    const Tensor* b = args[2] == Py_None ? nullptr : tensor(args[2]);
    if (!x || !w || (args[2] != Py_None && !b) || x->dim() != 2 || !real(x->scalar_type()) ||
        !PyFloat_Check(args[3]))
      Py_RETURN_NONE;
    const int64_t M = x->size(0), N = x->size(1);
    Call c(*x);
    c.need(*x, x->scalar_type(), {M, N});
    c.need(*w, at::kFloat, {N});
    if (b) c.need(*b, at::kFloat, {N});
    const int out = (int)PyLong_AsLong(args[4]);
    bool codes;
    if (!truth(args[5], codes)) return nullptr;
    if (!c.ok || N < 1 || N > 16384 || (codes ? N % 128 != 0 : out < 0)) Py_RETURN_NONE;
    Tensor y, q, s;
    if (out >= 0) y = c.make(out_type(out), {M, N});
    if (codes) {
      q = c.make(at::kByte, {M, N});
      s = c.make(at::kFloat, {N / 128, M});
    }
    const Tensor mean = c.make(at::kFloat, {M}), rstd = c.make(at::kFloat, {M});
    const fp8q_status st = entries.layer_norm(
        at_(*x), type_code(x->scalar_type()), at_<float>(*w), b ? at_<float>(*b) : nullptr, M, N,
        (float)PyFloat_AS_DOUBLE(args[3]), at_(y),
        out == FP8Q_OUT_BF16 ? FP8Q_OUT_BF16 : FP8Q_OUT_F32, at_<uint8_t>(q), at_<float>(s),
        (fp8q_scale_mode)PyLong_AsLong(args[6]), at_<float>(mean), at_<float>(rstd), c.stream());
    if (!codes) return answers(st, y, mean, rstd);
    return y.defined() ? answers(st, q, s, mean, rstd, y) : answers(st, q, s, mean, rstd);
  });
}

// layer_norm_backward(dy, x, weight, mean, rstd, bias)
PyObject* layer_norm_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS(6)
  return guarded([&]() -> PyObject* {
    const Tensor *dy = tensor(args[0]), *x = tensor(args[1]), *w = tensor(args[2]),
                 *mean = tensor(args[3]), *rstd = tensor(args[4]);
    if (!dy || !x || !w || !mean || !rstd || x->dim() != 2 || !real(x->scalar_type()) ||
        !real(dy->scalar_type()))
      Py_RETURN_NONE;
    const int64_t M = x->size(0), N = x->size(1);
    Call c(*x);
    c.need(*x, x->scalar_type(), {M, N});
    c.need(*dy, dy->scalar_type(), {M, N});
    c.need(*w, at::kFloat, {N});
    c.need(*mean, at::kFloat, {M});
    c.need(*rstd, at::kFloat, {M});
    bool bias;
    if (!truth(args[5], bias)) return nullptr;
    if (!c.ok || N < 1 || N > 16384) Py_RETURN_NONE;
    const Tensor dx = c.make(x->scalar_type(), {M, N}), dw = c.make(at::kFloat, {N});
    const Tensor db = bias ? c.make(at::kFloat, {N}) : Tensor();
    const Tensor work = c.make(at::kByte, {entries.layer_norm_backward_workspace(M, N)});
    return answers(entries.layer_norm_backward(
                       at_(*dy), type_code(dy->scalar_type()), at_(*x),
                       type_code(x->scalar_type()), at_<float>(*w), at_<float>(*mean),
                       at_<float>(*rstd), M, N, at_(dx), at_<float>(dw), at_<float>(db), at_(work),
                       c.stream()),
                   dx, dw, db);
  });
}

// The experts of a device off [G + 1], or 0 where it is none.
int32_t experts(const Tensor* off, Call& c) {
  if (!off || off->dim() != 1 || off->size(0) < 2 || off->size(0) > 1025) return 0;
  c.need(*off, at::kInt, {off->size(0)});
  return (int32_t)off->size(0) - 1;
}

// grouped_quantize_act_t(x, off, mode)
PyObject* grouped_quantize_act_t(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS(3)
  return guarded([&]() -> PyObject* {
    const Tensor *x = tensor(args[0]), *off = tensor(args[1]);
    if (!x || x->dim() != 2) Py_RETURN_NONE;
    const int64_t M = x->size(0), K = x->size(1);
    Call c(*x);
    c.need(*x, at::kBFloat16, {M, K});
    const int32_t G = experts(off, c);
    if (!c.ok || !G || K % 128) Py_RETURN_NONE;
    const int64_t T = entries.expert_columns(M, G);
    const Tensor q = c.make(at::kByte, {K, T}), s = c.make(at::kFloat, {T / 128, K});
    return answers(entries.grouped_quantize_act_t(at_(*x), M, at_<int32_t>(*off), G, K,
                                                  at_<uint8_t>(q), at_<float>(s),
                                                  (fp8q_scale_mode)PyLong_AsLong(args[2]),
                                                  c.stream()),
                   q, s);
  });
}

// grouped_gated_backward(dh, gate_up, off, act, mode, rows, tokens)
PyObject* grouped_gated_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS(7)
  return guarded([&]() -> PyObject* {
    const Tensor *dh = tensor(args[0]), *gu = tensor(args[1]), *off = tensor(args[2]);
    if (!dh || !gu || dh->dim() != 2) Py_RETURN_NONE;
    const int64_t M = dh->size(0), F = dh->size(1);
    Call c(*dh);
    c.need(*dh, at::kBFloat16, {M, F});
    c.need(*gu, at::kBFloat16, {M, 2 * F});
    const int32_t G = experts(off, c);
    bool rows, tokens;
    if (!truth(args[5], rows) || !truth(args[6], tokens)) return nullptr;
    if (!c.ok || !G || F % 128 || !(rows || tokens)) Py_RETURN_NONE;
    Tensor q, s, qt, st;
    if (rows) {
      q = c.make(at::kByte, {M, 2 * F});
      s = c.make(at::kFloat, {2 * F / 128, M});
    }
    if (tokens) {
      const int64_t T = entries.expert_columns(M, G);
      qt = c.make(at::kByte, {2 * F, T});
      st = c.make(at::kFloat, {T / 128, 2 * F});
    }
    return answers(entries.grouped_gated_backward(
                       at_(*dh), at_(*gu), M, at_<int32_t>(*off), G, F,
                       (fp8q_activation)PyLong_AsLong(args[3]),
                       (fp8q_scale_mode)PyLong_AsLong(args[4]), at_<uint8_t>(q), at_<float>(s),
                       at_<uint8_t>(qt), at_<float>(st), c.stream()),
                   q, s, qt, st);
  });
}

// grouped_gemm_rowscaled(a_q, a_s, b_q, b_s, off, out, precise)
PyObject* grouped_gemm_rowscaled(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS(7)
  return guarded([&]() -> PyObject* {
    const Tensor *a = tensor(args[0]), *as = tensor(args[1]), *b = tensor(args[2]),
                 *bs = tensor(args[3]), *off = tensor(args[4]);
    if (!a || !as || !b || !bs || a->dim() != 2 || b->dim() != 2) Py_RETURN_NONE;
    const int64_t N = a->size(0), T = a->size(1), K = b->size(0);
    Call c(*a);
    c.need(*a, at::kByte, {N, T});
    c.need(*as, at::kFloat, {T / 128, N});
    c.need(*b, at::kByte, {K, T});
    c.need(*bs, at::kFloat, {T / 128, K});
    const int32_t G = experts(off, c);
    bool precise;
    if (!truth(args[6], precise)) return nullptr;
    if (!c.ok || !G || N % 128 || K % 128 || T % 128) Py_RETURN_NONE;
    const int out = (int)PyLong_AsLong(args[5]);
    const Tensor w = c.make(out_type(out), {G, N, K});
    auto f = precise ? entries.grouped_gemm_rowscaled_precise : entries.grouped_gemm_rowscaled;
    return answer(f(at_<uint8_t>(*a), at_<float>(*as), at_<uint8_t>(*b), at_<float>(*bs), T,
                    at_<int32_t>(*off), G, N, K, at_(w), (fp8q_out_dtype)out, c.stream()),
                  w);
  });
}

// A list or tuple of `n` objects (any number where n < 0), or None: items NULL.
struct Items {
  PyObject** at = nullptr;
  Py_ssize_t n = 0;
  bool ok = true;
  Items(PyObject* o, Py_ssize_t want, bool optional) {
    if (optional && o == Py_None) return;
    ok = PyList_Check(o) || PyTuple_Check(o);
    if (!ok) return;
    n = PySequence_Fast_GET_SIZE(o);
    at = PySequence_Fast_ITEMS(o);
    ok = want < 0 || n == want;
  }
};

// A device tensor of one element; NULL where o is none.
const Tensor* device_scalar(PyObject* o, at::ScalarType type, Call& c) {
  const Tensor* t = tensor(o);
  if (!t || t->numel() != 1) return nullptr;
  c.need(*t, type, t->sizes());
  return t;
}

// adamw(params, grads, m, m_s, v, v_s, copies, step, lr, beta1, beta2, eps,
// weight_decay, grad_scale): the status.  The lists of scales and copies may be None.
PyObject* adamw(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS(14)
  return guarded([&]() -> PyObject* {
    const Items p(args[0], -1, false), g(args[1], p.n, false), m(args[2], p.n, false),
        ms(args[3], p.n, true), v(args[4], p.n, false), vs(args[5], p.n, true),
        copies(args[6], p.n, true);
    if (!p.ok || !g.ok || !m.ok || !ms.ok || !v.ok || !vs.ok || !copies.ok || p.n == 0 ||
        p.n > INT32_MAX || !ms.at != !vs.at)
      Py_RETURN_NONE;
    const Tensor *first = tensor(p.at[0]), *grad = tensor(g.at[0]);
    if (!first || !grad || !real(grad->scalar_type())) Py_RETURN_NONE;
    const auto moment = ms.at ? at::kByte : at::kFloat;
    Call c(*first);
    std::vector<fp8q_adamw_tensor> list((size_t)p.n);
    for (Py_ssize_t i = 0; i < p.n && c.ok; ++i) {
      const Tensor *tp = tensor(p.at[i]), *tg = tensor(g.at[i]), *tm = tensor(m.at[i]),
                   *tv = tensor(v.at[i]);
      if (!tp || !tg || !tm || !tv) Py_RETURN_NONE;
      const auto shape = tp->sizes();
      c.need(*tp, at::kFloat, shape);
      c.need(*tg, grad->scalar_type(), shape);
      c.need(*tm, moment, shape);
      c.need(*tv, moment, shape);
      fp8q_adamw_tensor& t = list[(size_t)i];
      t = {at_<float>(*tp), at_(*tg), at_(*tm), at_(*tv), nullptr, nullptr, nullptr, tp->numel()};
      if (ms.at) {
        const Tensor *a = tensor(ms.at[i]), *b = tensor(vs.at[i]);
        if (!a || !b) Py_RETURN_NONE;
        c.need(*a, at::kFloat, {(t.n + 127) / 128});
        c.need(*b, at::kFloat, {(t.n + 127) / 128});
        t.m_s = at_<float>(*a);
        t.v_s = at_<float>(*b);
      }
      if (copies.at) {
        const Tensor* y = tensor(copies.at[i]);
        if (!y) Py_RETURN_NONE;
        c.need(*y, at::kBFloat16, shape);
        t.copy = at_(*y);
      }
    }
    fp8q_adamw_args a = {};
    if (PyLong_Check(args[7])) {
      a.step = PyLong_AsLongLong(args[7]);
      if (a.step == -1 && PyErr_Occurred()) return nullptr;
    } else if (const Tensor* t = device_scalar(args[7], at::kInt, c)) {
      a.step_dev = at_<int32_t>(*t);
    } else {
      Py_RETURN_NONE;
    }
    if (PyFloat_Check(args[8])) {
      a.lr = PyFloat_AS_DOUBLE(args[8]);
    } else if (const Tensor* t = device_scalar(args[8], at::kFloat, c)) {
      a.lr_dev = at_<float>(*t);
    } else {
      Py_RETURN_NONE;
    }
    for (int i = 9; i < 13; ++i)
      if (!PyFloat_Check(args[i])) Py_RETURN_NONE;
    a.beta1 = PyFloat_AS_DOUBLE(args[9]);
    a.beta2 = PyFloat_AS_DOUBLE(args[10]);
    a.eps = PyFloat_AS_DOUBLE(args[11]);
    a.weight_decay = PyFloat_AS_DOUBLE(args[12]);
    if (args[13] != Py_None) {
      const Tensor* t = device_scalar(args[13], at::kFloat, c);
      if (!t) Py_RETURN_NONE;
      a.grad_scale = at_<float>(*t);
    }
    // (values out of range: the Python path says which)
    auto bad = [](double x, double end) { return !(x >= 0.0 && x < end); };
    if (!c.ok || bad(a.lr, INFINITY) || bad(a.beta1, 1) || bad(a.beta2, 1) ||
        (a.eps != 0.0 && !(a.eps >= 0x1p-126 && a.eps <= 0x1p125)) ||
        bad(a.weight_decay, INFINITY) || (!a.step_dev && a.step < 1))
      Py_RETURN_NONE;
    const fp8q_status st =
        entries.adamw(list.data(), (int32_t)p.n, &a, type_code(grad->scalar_type()),
                      ms.at ? FP8Q_MOMENTS_E4M3 : FP8Q_MOMENTS_F32, c.stream());
    if (st == FP8Q_OK)  // autograd hears of what was written
      for (const Items* l : {&p, &m, &v, &ms, &vs, &copies})
        for (Py_ssize_t i = 0; l->at && i < l->n; ++i) {
          const Tensor& t = THPVariable_Unpack(l->at[i]);
          if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
        }
    return PyLong_FromLong(st);
  });
}

// entries(address, ...): the C entry points, in the order of Entries
PyObject* set_entries(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  NEEDS((int)kEntries)
  void* at[kEntries];
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
    at[i] = PyLong_AsVoidPtr(args[i]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a NULL entry point");
      return nullptr;
    }
  }
  memcpy(&entries, at, sizeof entries);
  Py_RETURN_NONE;
}

#define METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(quantize_token_i8), METHOD(gemm_i8), METHOD(gemm_i8_gated),
                         METHOD(gemm_gated), METHOD(gated_backward), METHOD(layer_norm),
                         METHOD(layer_norm_backward), METHOD(grouped_quantize_act_t),
                         METHOD(grouped_gated_backward), METHOD(grouped_gemm_rowscaled),
                         METHOD(adamw),
                         {"entries", (PyCFunction)(void (*)(void))set_entries, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
