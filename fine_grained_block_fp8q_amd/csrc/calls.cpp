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
                         METHOD(gemm_gated), METHOD(gated_backward),
                         {"entries", (PyCFunction)(void (*)(void))set_entries, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
