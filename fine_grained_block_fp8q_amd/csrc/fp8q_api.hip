// C ABI of libfp8q: host-side validation and launch (declared in include/fp8q.h).
//
// Validation runs entirely on the host and before any HIP call, in the order
// the header documents, so every error path can be exercised without a GPU.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>

#include "fp8q.h"

namespace fp8q {
hipError_t launch_quantize_act(const void* x, int64_t M, int64_t K, uint8_t* q, float* s,
                               int mode, hipStream_t stream);
hipError_t launch_quantize_weight(const void* w, int64_t N, int64_t K, uint8_t* q, float* s,
                                  int mode, hipStream_t stream);
hipError_t launch_gemm(const uint8_t* a_q, const float* a_s, const uint8_t* w_q,
                       const float* w_s, int64_t M, int64_t N, int64_t K, void* c, int out_bf16,
                       int mode, hipStream_t stream);
hipError_t launch_grouped_gemm(const uint8_t* a_q, const float* a_s, int64_t M_total,
                               const int32_t* off, int G, const uint8_t* w_q, const float* w_s,
                               int64_t N, int64_t K, void* c, int out_bf16, int precise,
                               hipStream_t stream);
hipError_t launch_gemm_bf16(const void* a, const void* w, int64_t M, int64_t N, int64_t K,
                            void* c, int out_bf16, hipStream_t stream);
hipError_t launch_quantize_act_t(const void* x, int64_t M, int64_t K, uint8_t* qt, float* st,
                                 int mode, hipStream_t stream);
hipError_t launch_quantize_weight_t(const void* w, int64_t N, int64_t K, uint8_t* qt,
                                    float* st, int mode, hipStream_t stream);
hipError_t launch_gemm_rowscaled(const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                                 const float* b_s, int64_t M, int64_t N, int64_t K, void* c,
                                 int out_bf16, int precise, hipStream_t stream);
hipError_t launch_gemm_cast(const void* x, const uint8_t* w_q, const float* w_s, int64_t M,
                            int64_t N, int64_t K, void* c, int out_bf16, int mode,
                            hipStream_t stream);
hipError_t launch_grouped_gemm_cast(const void* x, int64_t M_total, const int32_t* off, int G,
                                    const uint8_t* w_q, const float* w_s, int64_t N, int64_t K,
                                    void* c, int out_bf16, int mode, hipStream_t stream);
hipError_t launch_quantize_token_i8(const void* x, int64_t M, int64_t K, int64_t Kp, int8_t* q,
                                    float* s, hipStream_t stream);
hipError_t launch_gemm_i8(const int8_t* a_q, const float* a_s, const int8_t* w_q, const float* w_s,
                          const float* bias, int64_t M, int64_t N, int64_t K, void* c,
                          int out_bf16, hipStream_t stream);
hipError_t launch_gemm_i8_gated(const int8_t* a_q, const float* a_s, const int8_t* w_q,
                                const float* w_s, int64_t M, int64_t F, int64_t K, int act,
                                void* h, int out_bf16, hipStream_t stream);
hipError_t launch_gemm_gated(const uint8_t* a_q, const float* a_s, int64_t M, const int32_t* off,
                             int G, const uint8_t* w_q, const float* w_s, int64_t F, int64_t K,
                             int act, void* h, int out_bf16, void* gu, hipStream_t stream);
hipError_t launch_gated_backward(const void* dh, const void* gu, int64_t M, int64_t F, int act,
                                 int mode, uint8_t* q, float* s, uint8_t* qt, float* st,
                                 hipStream_t stream);
hipError_t launch_layer_norm(const void* x, int x_bf16, const float* weight, const float* bias,
                             int64_t M, int64_t N, float eps, void* y, int y_bf16, uint8_t* q,
                             float* s, int mode, float* mean, float* rstd, hipStream_t stream);
int64_t layer_norm_backward_workspace(int64_t M, int64_t N);
hipError_t launch_layer_norm_backward(const void* dy, int dy_bf16, const void* x, int x_bf16,
                                      const float* weight, const float* mean, const float* rstd,
                                      int64_t M, int64_t N, void* dx, float* dweight, float* dbias,
                                      float* workspace, hipStream_t stream);
int64_t expert_columns(int64_t M, int64_t G);
hipError_t launch_grouped_quantize_act_t(const void* x, int64_t M, int64_t K, const int32_t* off,
                                         int G, uint8_t* qt, float* st, int mode,
                                         hipStream_t stream);
hipError_t launch_grouped_gated_backward(const void* dh, const void* gu, int64_t M,
                                         const int32_t* off, int G, int64_t F, int act, int mode,
                                         uint8_t* q, float* s, uint8_t* qt, float* st,
                                         hipStream_t stream);
hipError_t launch_grouped_gemm_rowscaled(const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                                         const float* b_s, int64_t T, const int32_t* off, int G,
                                         int64_t N, int64_t K, void* c, int out_bf16, int precise,
                                         hipStream_t stream);
hipError_t launch_adamw(const fp8q_adamw_tensor* tensors, int32_t count, const fp8q_adamw_args& h,
                        int grad_bf16, int e4m3, hipStream_t stream);
#ifdef FP8Q_DEBUG_CHECKS
hipError_t wgrad_offsets_error_take(hipStream_t stream, int* flag);
hipError_t tokens_offsets_error_take(hipStream_t stream, int* flag);
hipError_t backward_offsets_error_take(hipStream_t stream, int* flag);
hipError_t offsets_error_take(hipStream_t stream, int* flag);
hipError_t gated_offsets_error_take(hipStream_t stream, int* flag);
#endif
}  // namespace fp8q

namespace {

constexpr int kMaxDevices = 64;
// 0 = unknown, 1 = gfx950, 2 = other architecture
std::atomic<int> g_arch_cache[kMaxDevices];

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The current device must be a gfx950.  Cached per device ordinal.
fp8q_status check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    return FP8Q_ERR_DEVICE;
  }
  if (dev < kMaxDevices) {
    const int c = g_arch_cache[dev].load(std::memory_order_relaxed);
    if (c == 1) return FP8Q_OK;
    if (c == 2) return FP8Q_ERR_DEVICE;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
    (void)hipGetLastError();
    return FP8Q_ERR_DEVICE;
  }
  const bool ok = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < kMaxDevices) g_arch_cache[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? FP8Q_OK : FP8Q_ERR_DEVICE;
}

fp8q_status launched(hipError_t e) {
  if (e == hipSuccess) return FP8Q_OK;
  (void)hipGetLastError();
  return FP8Q_ERR_LAUNCH;
}

// A grouped launch's status.  Debug builds (FP8Q_DEBUG_CHECKS) synchronize
// the stream and report the verdict of kernel family `k` on the device offsets.
enum Grouped { kGrouped, kGated, kWgrad, kTokens, kBackward };

fp8q_status grouped_launched(hipError_t e, hipStream_t stream, Grouped k = kGrouped) {
  const fp8q_status st = launched(e);
#ifdef FP8Q_DEBUG_CHECKS
  if (st == FP8Q_OK) {
    int flag = 0;
    auto take = k == kGated      ? fp8q::gated_offsets_error_take
                : k == kWgrad    ? fp8q::wgrad_offsets_error_take
                : k == kTokens   ? fp8q::tokens_offsets_error_take
                : k == kBackward ? fp8q::backward_offsets_error_take
                                 : fp8q::offsets_error_take;
    if (take(stream, &flag) != hipSuccess) return launched(hipErrorUnknown);
    if (flag) return FP8Q_ERR_OFFSETS;
  }
#else
  (void)stream;
  (void)k;
#endif
  return st;
}

bool valid_mode(int m) { return m == FP8Q_SCALE_F32 || m == FP8Q_SCALE_POW2; }
bool valid_act(int a) { return a == FP8Q_ACT_SILU || a == FP8Q_ACT_GELU_TANH; }
bool valid_out(int o) { return o == FP8Q_OUT_F32 || o == FP8Q_OUT_BF16; }

}  // namespace

extern "C" {

int fp8q_abi_version(void) { return FP8Q_ABI_VERSION; }

int fp8q_debug_checks(void) {
#ifdef FP8Q_DEBUG_CHECKS
  return 1;
#else
  return 0;
#endif
}

const char* fp8q_status_string(fp8q_status st) {
  switch (st) {
    case FP8Q_OK: return "FP8Q_OK";
    case FP8Q_ERR_NULL: return "FP8Q_ERR_NULL: a required pointer is NULL";
    case FP8Q_ERR_SHAPE:
      return "FP8Q_ERR_SHAPE: negative size, K or N not a multiple of 128, or G < 1";
    case FP8Q_ERR_ALIGN:
      return "FP8Q_ERR_ALIGN: data pointer not 16-byte aligned or scale/offset pointer not "
             "4-byte aligned";
    case FP8Q_ERR_ENUM: return "FP8Q_ERR_ENUM: unknown scale mode or output dtype";
    case FP8Q_ERR_DEVICE: return "FP8Q_ERR_DEVICE: no current HIP device, or it is not gfx950";
    case FP8Q_ERR_LAUNCH: return "FP8Q_ERR_LAUNCH: kernel launch failed";
    case FP8Q_ERR_UNSUPPORTED: return "FP8Q_ERR_UNSUPPORTED: valid request outside what the library implements";
    case FP8Q_ERR_OFFSETS:
      return "FP8Q_ERR_OFFSETS: device offsets not 0 = off[0] <= ... <= off[G] <= M_total "
             "(reported by FP8Q_DEBUG_CHECKS builds)";
  }
  return "FP8Q_ERR_UNKNOWN: not a status code";
}

fp8q_status fp8q_quantize_act(const void* x_bf16, int64_t M, int64_t K, uint8_t* q, float* s,
                              fp8q_scale_mode mode, hipStream_t stream) {
  const bool empty = (M == 0 || K == 0);
  if (!empty && (!x_bf16 || !q || !s)) return FP8Q_ERR_NULL;
  if (M < 0 || K < 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(s, 4)) return FP8Q_ERR_ALIGN;
  if (!valid_mode(mode)) return FP8Q_ERR_ENUM;
  if (empty) return FP8Q_OK;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(fp8q::launch_quantize_act(x_bf16, M, K, q, s, (int)mode, stream));
}

fp8q_status fp8q_quantize_weight(const void* w_bf16, int64_t N, int64_t K, uint8_t* q, float* s,
                                 fp8q_scale_mode mode, hipStream_t stream) {
  const bool empty = (N == 0 || K == 0);
  if (!empty && (!w_bf16 || !q || !s)) return FP8Q_ERR_NULL;
  if (N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (!aligned(w_bf16, 16) || !aligned(q, 16) || !aligned(s, 4)) return FP8Q_ERR_ALIGN;
  if (!valid_mode(mode)) return FP8Q_ERR_ENUM;
  if (empty) return FP8Q_OK;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(fp8q::launch_quantize_weight(w_bf16, N, K, q, s, (int)mode, stream));
}

// The GEMM kernels address a tile's operands with 32-bit buffer offsets
// (row-in-tile * K + chunk offset) and a chunk's row scales with a 31-bit
// scalar offset (chunk * rows * 4): K up to 2^22 and rows * K/128 * 4 below
// 2^31 keep every offset in range.
static bool gemm_extent_ok(int64_t rows, int64_t K) {
  if (K > (int64_t(1) << 22)) return false;
  return rows <= int64_t(0x7FFFFFFF) / 4 / (K / 128);
}

static fp8q_status gemm_call(const uint8_t* a_q, const float* a_s, const uint8_t* w_q,
                             const float* w_s, int64_t M, int64_t N, int64_t K, void* c,
                             fp8q_out_dtype out, int mode, hipStream_t stream) {
  const bool empty_out = (M == 0 || N == 0);
  const bool empty_k = (K == 0);
  if (!empty_out && !c) return FP8Q_ERR_NULL;
  if (!empty_out && !empty_k && (!a_q || !a_s || !w_q || !w_s)) return FP8Q_ERR_NULL;
  if (M < 0 || N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (!aligned(a_q, 16) || !aligned(w_q, 16) || !aligned(c, 16) || !aligned(a_s, 4) ||
      !aligned(w_s, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_out(out)) return FP8Q_ERR_ENUM;
  if (empty_out) return FP8Q_OK;
  if (empty_k) return FP8Q_ERR_UNSUPPORTED;  // C = 0 would need a fill kernel
  if (!gemm_extent_ok(M, K)) return FP8Q_ERR_UNSUPPORTED;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(
      fp8q::launch_gemm(a_q, a_s, w_q, w_s, M, N, K, c, out == FP8Q_OUT_BF16, mode, stream));
}

fp8q_status fp8q_gemm(const uint8_t* a_q, const float* a_s, const uint8_t* w_q,
                      const float* w_s, int64_t M, int64_t N, int64_t K, void* c,
                      fp8q_out_dtype out, hipStream_t stream) {
  return gemm_call(a_q, a_s, w_q, w_s, M, N, K, c, out, 0, stream);
}

fp8q_status fp8q_gemm_precise(const uint8_t* a_q, const float* a_s, const uint8_t* w_q,
                              const float* w_s, int64_t M, int64_t N, int64_t K, void* c,
                              fp8q_out_dtype out, hipStream_t stream) {
  return gemm_call(a_q, a_s, w_q, w_s, M, N, K, c, out, 1, stream);
}

fp8q_status fp8q_gemm_mfma_scaled(const uint8_t* a_q, const float* a_s, const uint8_t* w_q,
                                  const float* w_s, int64_t M, int64_t N, int64_t K, void* c,
                                  fp8q_out_dtype out, hipStream_t stream) {
  return gemm_call(a_q, a_s, w_q, w_s, M, N, K, c, out, 2, stream);
}

static fp8q_status grouped_call(const uint8_t* a_q, const float* a_s, int64_t M_total,
                                const int32_t* off, int32_t G, const uint8_t* w_q,
                                const float* w_s, int64_t N, int64_t K, void* c,
                                fp8q_out_dtype out, int precise, hipStream_t stream) {
  const bool empty_out = (M_total == 0 || N == 0);
  if (!off) return FP8Q_ERR_NULL;
  if (!empty_out && !c) return FP8Q_ERR_NULL;
  if (!empty_out && K != 0 && (!a_q || !a_s || !w_q || !w_s)) return FP8Q_ERR_NULL;
  if (M_total < 0 || N < 0 || K < 0 || G < 1 || N % 128 != 0 || K % 128 != 0)
    return FP8Q_ERR_SHAPE;
  if (G > 1024) return FP8Q_ERR_UNSUPPORTED;
  if (M_total > 0x7FFFFFFF) return FP8Q_ERR_SHAPE;  // offsets are int32
  if (!aligned(a_q, 16) || !aligned(w_q, 16) || !aligned(c, 16) || !aligned(a_s, 4) ||
      !aligned(w_s, 4) || !aligned(off, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_out(out)) return FP8Q_ERR_ENUM;
  if (empty_out) return FP8Q_OK;
  if (K == 0) return FP8Q_ERR_UNSUPPORTED;
  if (!gemm_extent_ok(M_total, K)) return FP8Q_ERR_UNSUPPORTED;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return grouped_launched(fp8q::launch_grouped_gemm(a_q, a_s, M_total, off, G, w_q, w_s, N, K,
                                                    c, out == FP8Q_OUT_BF16, precise, stream),
                          stream);
}

fp8q_status fp8q_grouped_gemm(const uint8_t* a_q, const float* a_s, int64_t M_total,
                              const int32_t* off, int32_t G, const uint8_t* w_q,
                              const float* w_s, int64_t N, int64_t K, void* c,
                              fp8q_out_dtype out, hipStream_t stream) {
  return grouped_call(a_q, a_s, M_total, off, G, w_q, w_s, N, K, c, out, 0, stream);
}

fp8q_status fp8q_grouped_gemm_precise(const uint8_t* a_q, const float* a_s, int64_t M_total,
                                      const int32_t* off, int32_t G, const uint8_t* w_q,
                                      const float* w_s, int64_t N, int64_t K, void* c,
                                      fp8q_out_dtype out, hipStream_t stream) {
  return grouped_call(a_q, a_s, M_total, off, G, w_q, w_s, N, K, c, out, 1, stream);
}

fp8q_status fp8q_quantize_act_t(const void* x_bf16, int64_t M, int64_t K, uint8_t* q_t,
                                float* s_t, fp8q_scale_mode mode, hipStream_t stream) {
  const bool empty = (M == 0 || K == 0);
  if (!empty && (!x_bf16 || !q_t || !s_t)) return FP8Q_ERR_NULL;
  if (M < 0 || K < 0 || M % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(q_t, 16) || !aligned(s_t, 4)) return FP8Q_ERR_ALIGN;
  if (!valid_mode(mode)) return FP8Q_ERR_ENUM;
  if (empty) return FP8Q_OK;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(fp8q::launch_quantize_act_t(x_bf16, M, K, q_t, s_t, (int)mode, stream));
}

fp8q_status fp8q_quantize_weight_t(const void* w_bf16, int64_t N, int64_t K, uint8_t* q_t,
                                   float* s_t, fp8q_scale_mode mode, hipStream_t stream) {
  const bool empty = (N == 0 || K == 0);
  if (!empty && (!w_bf16 || !q_t || !s_t)) return FP8Q_ERR_NULL;
  if (N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (!aligned(w_bf16, 16) || !aligned(q_t, 16) || !aligned(s_t, 4)) return FP8Q_ERR_ALIGN;
  if (!valid_mode(mode)) return FP8Q_ERR_ENUM;
  if (empty) return FP8Q_OK;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(fp8q::launch_quantize_weight_t(w_bf16, N, K, q_t, s_t, (int)mode, stream));
}

static fp8q_status rowscaled_call(const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                                  const float* b_s, int64_t M, int64_t N, int64_t K, void* c,
                                  fp8q_out_dtype out, int precise, hipStream_t stream) {
  const bool empty_out = (M == 0 || N == 0);
  if (!empty_out && !c) return FP8Q_ERR_NULL;
  if (!empty_out && K != 0 && (!a_q || !a_s || !b_q || !b_s)) return FP8Q_ERR_NULL;
  if (M < 0 || N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(c, 16) || !aligned(a_s, 4) ||
      !aligned(b_s, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_out(out)) return FP8Q_ERR_ENUM;
  if (empty_out) return FP8Q_OK;
  if (K == 0) return FP8Q_ERR_UNSUPPORTED;
  if (!gemm_extent_ok(M, K) || !gemm_extent_ok(N, K)) return FP8Q_ERR_UNSUPPORTED;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(fp8q::launch_gemm_rowscaled(a_q, a_s, b_q, b_s, M, N, K, c,
                                              out == FP8Q_OUT_BF16, precise, stream));
}

fp8q_status fp8q_gemm_rowscaled(const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                                const float* b_s, int64_t M, int64_t N, int64_t K, void* c,
                                fp8q_out_dtype out, hipStream_t stream) {
  return rowscaled_call(a_q, a_s, b_q, b_s, M, N, K, c, out, 0, stream);
}

fp8q_status fp8q_gemm_rowscaled_precise(const uint8_t* a_q, const float* a_s,
                                        const uint8_t* b_q, const float* b_s, int64_t M,
                                        int64_t N, int64_t K, void* c, fp8q_out_dtype out,
                                        hipStream_t stream) {
  return rowscaled_call(a_q, a_s, b_q, b_s, M, N, K, c, out, 1, stream);
}

fp8q_status fp8q_gemm_bf16(const void* a, const void* w, int64_t M, int64_t N, int64_t K,
                           void* c, fp8q_out_dtype out, hipStream_t stream) {
  const bool empty_out = (M == 0 || N == 0);
  if (!empty_out && !c) return FP8Q_ERR_NULL;
  if (!empty_out && K != 0 && (!a || !w)) return FP8Q_ERR_NULL;
  if (M < 0 || N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(c, 16)) return FP8Q_ERR_ALIGN;
  if (!valid_out(out)) return FP8Q_ERR_ENUM;
  if (empty_out) return FP8Q_OK;
  if (K == 0) return FP8Q_ERR_UNSUPPORTED;
  if (K > (int64_t(1) << 21)) return FP8Q_ERR_UNSUPPORTED;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(fp8q::launch_gemm_bf16(a, w, M, N, K, c, out == FP8Q_OUT_BF16, stream));
}

// The fused GEMMs read 2K-byte BF16 activation rows through 32-bit buffer
// offsets (row-in-tile * 2K): K up to 2^21, as for the BF16 GEMM.
fp8q_status fp8q_gemm_fused(const void* x_bf16, const uint8_t* w_q, const float* w_s,
                            int64_t M, int64_t N, int64_t K, void* c, fp8q_out_dtype out,
                            fp8q_scale_mode mode, hipStream_t stream) {
  const bool empty_out = (M == 0 || N == 0);
  if (!empty_out && !c) return FP8Q_ERR_NULL;
  if (!empty_out && K != 0 && (!x_bf16 || !w_q || !w_s)) return FP8Q_ERR_NULL;
  if (M < 0 || N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(w_q, 16) || !aligned(c, 16) || !aligned(w_s, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_out(out) || !valid_mode(mode)) return FP8Q_ERR_ENUM;
  if (empty_out) return FP8Q_OK;
  if (K == 0) return FP8Q_ERR_UNSUPPORTED;
  if (K > (int64_t(1) << 21)) return FP8Q_ERR_UNSUPPORTED;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(fp8q::launch_gemm_cast(x_bf16, w_q, w_s, M, N, K, c, out == FP8Q_OUT_BF16,
                                         (int)mode, stream));
}

fp8q_status fp8q_grouped_gemm_fused(const void* x_bf16, int64_t M_total, const int32_t* off,
                                    int32_t G, const uint8_t* w_q, const float* w_s, int64_t N,
                                    int64_t K, void* c, fp8q_out_dtype out, fp8q_scale_mode mode,
                                    hipStream_t stream) {
  const bool empty_out = (M_total == 0 || N == 0);
  if (!off) return FP8Q_ERR_NULL;
  if (!empty_out && !c) return FP8Q_ERR_NULL;
  if (!empty_out && K != 0 && (!x_bf16 || !w_q || !w_s)) return FP8Q_ERR_NULL;
  if (M_total < 0 || N < 0 || K < 0 || G < 1 || N % 128 != 0 || K % 128 != 0)
    return FP8Q_ERR_SHAPE;
  if (G > 1024) return FP8Q_ERR_UNSUPPORTED;
  if (M_total > 0x7FFFFFFF) return FP8Q_ERR_SHAPE;  // offsets are int32
  if (!aligned(x_bf16, 16) || !aligned(w_q, 16) || !aligned(c, 16) || !aligned(w_s, 4) ||
      !aligned(off, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_out(out) || !valid_mode(mode)) return FP8Q_ERR_ENUM;
  if (empty_out) return FP8Q_OK;
  if (K == 0) return FP8Q_ERR_UNSUPPORTED;
  if (K > (int64_t(1) << 21)) return FP8Q_ERR_UNSUPPORTED;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return grouped_launched(fp8q::launch_grouped_gemm_cast(x_bf16, M_total, off, G, w_q, w_s, N,
                                                         K, c, out == FP8Q_OUT_BF16, (int)mode,
                                                         stream),
                          stream);
}

fp8q_status fp8q_quantize_token_i8(const void* x_bf16, int64_t M, int64_t K, int8_t* q, float* s,
                                   hipStream_t stream) {
  const bool empty = M == 0;
  if (!empty && (!s || (K != 0 && (!x_bf16 || !q)))) return FP8Q_ERR_NULL;
  if (M < 0 || K < 0) return FP8Q_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(s, 4)) return FP8Q_ERR_ALIGN;
  if (empty) return FP8Q_OK;
  if (K == 0) return FP8Q_ERR_UNSUPPORTED;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(
      fp8q::launch_quantize_token_i8(x_bf16, M, K, (K + 15) / 16 * 16, q, s, stream));
}

// Checks shared by the int8 products: `out_cols` output columns, `w_rows`
// weight rows.  FP8Q_OK with *done set means there is nothing to compute.
static fp8q_status i8_args(const int8_t* a_q, const float* a_s, const int8_t* w_q,
                           const float* w_s, const float* bias, int64_t M, int64_t out_cols,
                           int64_t K, const void* c, int out, bool* done) {
  const bool empty_out = (M == 0 || out_cols == 0);
  *done = true;
  if (!empty_out && !c) return FP8Q_ERR_NULL;
  if (!empty_out && K != 0 && (!a_q || !a_s || !w_q || !w_s)) return FP8Q_ERR_NULL;
  if (M < 0 || out_cols < 0 || K < 0 || K % 16 != 0) return FP8Q_ERR_SHAPE;
  if (!aligned(a_q, 16) || !aligned(w_q, 16) || !aligned(c, 16) || !aligned(a_s, 4) ||
      !aligned(w_s, 4) || !aligned(bias, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_out(out)) return FP8Q_ERR_ENUM;
  if (empty_out) return FP8Q_OK;
  // 128 * 128 * K must stay below 2^31; K == 0 would need a fill kernel
  if (K == 0 || K >= 131072) return FP8Q_ERR_UNSUPPORTED;
  *done = false;
  return FP8Q_OK;
}

fp8q_status fp8q_gemm_i8(const int8_t* a_q, const float* a_s, const int8_t* w_q, const float* w_s,
                         const float* bias, int64_t M, int64_t N, int64_t K, void* c,
                         fp8q_out_dtype out, hipStream_t stream) {
  bool done;
  fp8q_status st = i8_args(a_q, a_s, w_q, w_s, bias, M, N, K, c, out, &done);
  if (st != FP8Q_OK || done) return st;
  st = check_device();
  if (st != FP8Q_OK) return st;
  return launched(fp8q::launch_gemm_i8(a_q, a_s, w_q, w_s, bias, M, N, K, c,
                                       out == FP8Q_OUT_BF16, stream));
}

fp8q_status fp8q_gemm_i8_gated(const int8_t* a_q, const float* a_s, const int8_t* w_q,
                               const float* w_s, int64_t M, int64_t F, int64_t K,
                               fp8q_activation act, void* h, fp8q_out_dtype out,
                               hipStream_t stream) {
  bool done;
  fp8q_status st = i8_args(a_q, a_s, w_q, w_s, nullptr, M, F, K, h, out, &done);
  if (st == FP8Q_OK && !valid_act(act)) st = FP8Q_ERR_ENUM;
  if (st != FP8Q_OK || done) return st;
  st = check_device();
  if (st != FP8Q_OK) return st;
  return launched(fp8q::launch_gemm_i8_gated(a_q, a_s, w_q, w_s, M, F, K, act, h,
                                             out == FP8Q_OUT_BF16, stream));
}

// off NULL and G 0: the dense call.
static fp8q_status gated_call(const uint8_t* a_q, const float* a_s, int64_t M, bool grouped,
                              const int32_t* off, int32_t G, const uint8_t* w_q, const float* w_s,
                              int64_t F, int64_t K, int act, void* h, int out, void* gate_up,
                              hipStream_t stream) {
  const bool empty_out = (M == 0 || F == 0);
  if (grouped && !off) return FP8Q_ERR_NULL;
  if (!empty_out && !h) return FP8Q_ERR_NULL;
  if (!empty_out && K != 0 && (!a_q || !a_s || !w_q || !w_s)) return FP8Q_ERR_NULL;
  if (M < 0 || F < 0 || K < 0 || F % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (grouped && (G < 1 || M > 0x7FFFFFFF)) return FP8Q_ERR_SHAPE;  // offsets are int32
  if (!aligned(a_q, 16) || !aligned(w_q, 16) || !aligned(h, 16) || !aligned(gate_up, 16) ||
      !aligned(a_s, 4) || !aligned(w_s, 4) || !aligned(off, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_act(act) || !valid_out(out)) return FP8Q_ERR_ENUM;
  if (grouped && G > 1024) return FP8Q_ERR_UNSUPPORTED;
  if (empty_out) return FP8Q_OK;
  if (K == 0 || !gemm_extent_ok(M, K)) return FP8Q_ERR_UNSUPPORTED;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  const hipError_t e = fp8q::launch_gemm_gated(a_q, a_s, M, off, G, w_q, w_s, F, K, act, h,
                                               out == FP8Q_OUT_BF16, gate_up, stream);
  return grouped ? grouped_launched(e, stream, kGated) : launched(e);
}

fp8q_status fp8q_gemm_gated(const uint8_t* a_q, const float* a_s, const uint8_t* w_q,
                            const float* w_s, int64_t M, int64_t F, int64_t K,
                            fp8q_activation act, void* h, fp8q_out_dtype out, void* gate_up,
                            hipStream_t stream) {
  return gated_call(a_q, a_s, M, false, nullptr, 0, w_q, w_s, F, K, act, h, out, gate_up, stream);
}

fp8q_status fp8q_grouped_gemm_gated(const uint8_t* a_q, const float* a_s, int64_t M_total,
                                    const int32_t* off, int32_t G, const uint8_t* w_q,
                                    const float* w_s, int64_t F, int64_t K, fp8q_activation act,
                                    void* h, fp8q_out_dtype out, void* gate_up,
                                    hipStream_t stream) {
  return gated_call(a_q, a_s, M_total, true, off, G, w_q, w_s, F, K, act, h, out, gate_up, stream);
}

fp8q_status fp8q_gated_backward(const void* dh, const void* gate_up, int64_t M, int64_t F,
                                fp8q_activation act, fp8q_scale_mode mode, uint8_t* q, float* s,
                                uint8_t* qt, float* st, hipStream_t stream) {
  const bool empty = (M == 0 || F == 0);
  if (!empty && (!dh || !gate_up || !q != !s || !qt != !st || (!q && !qt))) return FP8Q_ERR_NULL;
  if (M < 0 || F < 0 || F % 128 != 0) return FP8Q_ERR_SHAPE;
  if (!aligned(dh, 16) || !aligned(gate_up, 16) || !aligned(q, 16) || !aligned(qt, 16) ||
      !aligned(s, 4) || !aligned(st, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_act(act) || !valid_mode(mode)) return FP8Q_ERR_ENUM;
  if (empty) return FP8Q_OK;
  if (F > (int64_t(1) << 22)) return FP8Q_ERR_UNSUPPORTED;  // 32-bit offsets within 128 tokens
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(fp8q::launch_gated_backward(dh, gate_up, M, F, act, mode, q, s, qt, st, stream));
}

fp8q_status fp8q_layer_norm(const void* x, fp8q_out_dtype x_type, const float* weight,
                            const float* bias, int64_t M, int64_t N, float eps, void* y,
                            fp8q_out_dtype y_type, uint8_t* q, float* s, fp8q_scale_mode mode,
                            float* mean, float* rstd, hipStream_t stream) {
  const bool empty = M == 0;
  if (!empty && (!x || !weight || !mean || !rstd || !q != !s || (!y && !q))) return FP8Q_ERR_NULL;
  if (M < 0 || N < 1 || (q && N % 128 != 0)) return FP8Q_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(q, 16) || !aligned(weight, 4) ||
      !aligned(bias, 4) || !aligned(s, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_out(x_type) || !valid_out(y_type) || !valid_mode(mode)) return FP8Q_ERR_ENUM;
  if (N > 16384 || !(eps >= 0.f) || !isfinite(eps)) return FP8Q_ERR_UNSUPPORTED;
  if (empty) return FP8Q_OK;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(fp8q::launch_layer_norm(x, x_type == FP8Q_OUT_BF16, weight, bias, M, N, eps, y,
                                          y_type == FP8Q_OUT_BF16, q, s, mode, mean, rstd,
                                          stream));
}

int64_t fp8q_layer_norm_backward_workspace(int64_t M, int64_t N) {
  return M > 0 && N > 0 && N <= 16384 ? fp8q::layer_norm_backward_workspace(M, N) : 0;
}

fp8q_status fp8q_layer_norm_backward(const void* dy, fp8q_out_dtype dy_type, const void* x,
                                     fp8q_out_dtype x_type, const float* weight,
                                     const float* mean, const float* rstd, int64_t M, int64_t N,
                                     void* dx, float* dweight, float* dbias, void* workspace,
                                     hipStream_t stream) {
  if (!dweight) return FP8Q_ERR_NULL;
  if (M != 0 && (!dy || !x || !weight || !mean || !rstd || !dx)) return FP8Q_ERR_NULL;
  if (!workspace && fp8q_layer_norm_backward_workspace(M, N) != 0) return FP8Q_ERR_NULL;
  if (M < 0 || N < 1) return FP8Q_ERR_SHAPE;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dx, 16) || !aligned(workspace, 16) ||
      !aligned(weight, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) ||
      !aligned(dbias, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_out(dy_type) || !valid_out(x_type)) return FP8Q_ERR_ENUM;
  if (N > 16384) return FP8Q_ERR_UNSUPPORTED;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(fp8q::launch_layer_norm_backward(
      dy, dy_type == FP8Q_OUT_BF16, x, x_type == FP8Q_OUT_BF16, weight, mean, rstd, M, N, dx,
      dweight, dbias, static_cast<float*>(workspace), stream));
}

int64_t fp8q_expert_columns(int64_t M_total, int32_t G) {
  return M_total > 0 && G > 0 ? fp8q::expert_columns(M_total, G) : 0;
}

fp8q_status fp8q_grouped_quantize_act_t(const void* x_bf16, int64_t M_total, const int32_t* off,
                                        int32_t G, int64_t K, uint8_t* q_t, float* s_t,
                                        fp8q_scale_mode mode, hipStream_t stream) {
  const bool empty = (M_total == 0 || K == 0);
  if (!off || (!empty && (!x_bf16 || !q_t || !s_t))) return FP8Q_ERR_NULL;
  if (M_total < 0 || M_total > 0x7FFFFFFF || K < 0 || K % 128 != 0 || G < 1) return FP8Q_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(q_t, 16) || !aligned(s_t, 4) || !aligned(off, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_mode(mode)) return FP8Q_ERR_ENUM;
  if (G > 1024 || K > (int64_t(1) << 22)) return FP8Q_ERR_UNSUPPORTED;  // 32-bit offsets
  if (empty) return FP8Q_OK;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return grouped_launched(
      fp8q::launch_grouped_quantize_act_t(x_bf16, M_total, K, off, G, q_t, s_t, mode, stream),
      stream, kTokens);
}

fp8q_status fp8q_grouped_gated_backward(const void* dh, const void* gate_up, int64_t M_total,
                                        const int32_t* off, int32_t G, int64_t F,
                                        fp8q_activation act, fp8q_scale_mode mode, uint8_t* q,
                                        float* s, uint8_t* qt, float* st, hipStream_t stream) {
  const bool empty = (M_total == 0 || F == 0);
  if (!off || (!empty && (!dh || !gate_up || !q != !s || !qt != !st || (!q && !qt))))
    return FP8Q_ERR_NULL;
  if (M_total < 0 || M_total > 0x7FFFFFFF || F < 0 || F % 128 != 0 || G < 1) return FP8Q_ERR_SHAPE;
  if (!aligned(dh, 16) || !aligned(gate_up, 16) || !aligned(q, 16) || !aligned(qt, 16) ||
      !aligned(s, 4) || !aligned(st, 4) || !aligned(off, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_act(act) || !valid_mode(mode)) return FP8Q_ERR_ENUM;
  if (G > 1024 || F > (int64_t(1) << 22)) return FP8Q_ERR_UNSUPPORTED;  // 32-bit offsets
  if (empty) return FP8Q_OK;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return grouped_launched(fp8q::launch_grouped_gated_backward(dh, gate_up, M_total, off, G, F, act,
                                                              mode, q, s, qt, st, stream),
                          stream, kBackward);
}

static fp8q_status grouped_rowscaled_call(const uint8_t* a_q, const float* a_s,
                                          const uint8_t* b_q, const float* b_s, int64_t T,
                                          const int32_t* off, int32_t G, int64_t N, int64_t K,
                                          void* c, int out, int precise, hipStream_t stream) {
  const bool empty_out = (N == 0 || K == 0);
  if (!off || (!empty_out && !c)) return FP8Q_ERR_NULL;
  if (!empty_out && T != 0 && (!a_q || !a_s || !b_q || !b_s)) return FP8Q_ERR_NULL;
  if (T < 0 || N < 0 || K < 0 || T % 128 != 0 || N % 128 != 0 || K % 128 != 0 || G < 1)
    return FP8Q_ERR_SHAPE;
  if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(c, 16) || !aligned(a_s, 4) ||
      !aligned(b_s, 4) || !aligned(off, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_out(out)) return FP8Q_ERR_ENUM;
  // 32-bit offsets within a tile's rows of T bytes, and of 4 K bytes
  if (G > 1024 || T > (int64_t(1) << 24) || N > (int64_t(1) << 22) || K > (int64_t(1) << 22))
    return FP8Q_ERR_UNSUPPORTED;
  if (empty_out) return FP8Q_OK;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return grouped_launched(
      fp8q::launch_grouped_gemm_rowscaled(a_q, a_s, b_q, b_s, T, off, G, N, K, c,
                                          out == FP8Q_OUT_BF16, precise, stream),
      stream, kWgrad);
}

fp8q_status fp8q_grouped_gemm_rowscaled(const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                                        const float* b_s, int64_t T, const int32_t* off,
                                        int32_t G, int64_t N, int64_t K, void* c,
                                        fp8q_out_dtype out, hipStream_t stream) {
  return grouped_rowscaled_call(a_q, a_s, b_q, b_s, T, off, G, N, K, c, out, 0, stream);
}

fp8q_status fp8q_grouped_gemm_rowscaled_precise(const uint8_t* a_q, const float* a_s,
                                                const uint8_t* b_q, const float* b_s, int64_t T,
                                                const int32_t* off, int32_t G, int64_t N,
                                                int64_t K, void* c, fp8q_out_dtype out,
                                                hipStream_t stream) {
  return grouped_rowscaled_call(a_q, a_s, b_q, b_s, T, off, G, N, K, c, out, 1, stream);
}

// Whether two tensors' p overlap.  A list in the order of its addresses (views of one
// buffer) shows it at once; else a short one is compared pair by pair, a long one
// sorted.
static bool p_before(const fp8q_adamw_tensor* a, const fp8q_adamw_tensor* b) {
  return a->n == 0 || b->n == 0 || reinterpret_cast<uintptr_t>(a->p + a->n) <=
                                       reinterpret_cast<uintptr_t>(b->p);
}

static int by_p(const void* x, const void* y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>((*static_cast<const fp8q_adamw_tensor* const*>(x))->p);
  const uintptr_t b = reinterpret_cast<uintptr_t>((*static_cast<const fp8q_adamw_tensor* const*>(y))->p);
  return a < b ? -1 : a > b;
}

static fp8q_status check_overlap(const fp8q_adamw_tensor* t, int32_t count) {
  bool ordered = true;
  int32_t last = -1;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    ordered = ordered && (last < 0 || p_before(t + last, t + i));
    last = i;
  }
  if (ordered) return FP8Q_OK;
  if (count <= 64) {
    for (int32_t i = 1; i < count; ++i)
      for (int32_t j = 0; j < i; ++j)
        if (!p_before(t + i, t + j) && !p_before(t + j, t + i)) return FP8Q_ERR_UNSUPPORTED;
    return FP8Q_OK;
  }
  auto** order = static_cast<const fp8q_adamw_tensor**>(malloc(sizeof(void*) * (size_t)count));
  if (!order) return FP8Q_ERR_LAUNCH;
  int32_t n = 0;
  for (int32_t i = 0; i < count; ++i)
    if (t[i].n > 0) order[n++] = t + i;
  qsort(order, (size_t)n, sizeof *order, by_p);
  bool apart = true;
  for (int32_t i = 1; i < n; ++i) apart = apart && p_before(order[i - 1], order[i]);
  free(order);
  return apart ? FP8Q_OK : FP8Q_ERR_UNSUPPORTED;
}

static bool not_negative(double v) { return v >= 0.0 && isfinite(v); }

// The update's reciprocal takes denominators from 2^-126 to 2^126 (an eps below would be
// zero to it, and 0/0 of an element without a gradient; root terms stay below 2^92).
static bool usable_eps(double v) { return v == 0.0 || (v >= 0x1p-126 && v <= 0x1p125); }

fp8q_status fp8q_adamw(const fp8q_adamw_tensor* tensors, int32_t count,
                       const fp8q_adamw_args* args, fp8q_out_dtype grad_type,
                       fp8q_moments moments, hipStream_t stream) {
  const bool e4m3 = moments == FP8Q_MOMENTS_E4M3;
  if (!args || (count > 0 && !tensors)) return FP8Q_ERR_NULL;
  int64_t work = 0;
  for (int32_t i = 0; i < count; ++i) {
    const fp8q_adamw_tensor& t = tensors[i];
    if (t.n > 0 && (!t.p || !t.g || !t.m || !t.v || (e4m3 && (!t.m_s || !t.v_s))))
      return FP8Q_ERR_NULL;
  }
  if (count < 0) return FP8Q_ERR_SHAPE;
  for (int32_t i = 0; i < count; ++i)
    if (tensors[i].n < 0) return FP8Q_ERR_SHAPE;
  for (int32_t i = 0; i < count; ++i) {
    const fp8q_adamw_tensor& t = tensors[i];
    if (!aligned(t.p, 16) || !aligned(t.g, 16) || !aligned(t.m, 16) || !aligned(t.v, 16) ||
        !aligned(t.copy, 16) || !aligned(t.m_s, 4) || !aligned(t.v_s, 4))
      return FP8Q_ERR_ALIGN;
    work |= t.n;
  }
  if (!aligned(args->lr_dev, 4) || !aligned(args->step_dev, 4) || !aligned(args->grad_scale, 4))
    return FP8Q_ERR_ALIGN;
  if (!valid_out(grad_type) || (moments != FP8Q_MOMENTS_F32 && !e4m3)) return FP8Q_ERR_ENUM;
  if ((!args->lr_dev && !not_negative(args->lr)) || !usable_eps(args->eps) ||
      !not_negative(args->weight_decay) || !(args->beta1 >= 0.0 && args->beta1 < 1.0) ||
      !(args->beta2 >= 0.0 && args->beta2 < 1.0) || (!args->step_dev && args->step < 1))
    return FP8Q_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < count; ++i)
    if (tensors[i].n > (int64_t(1) << 34)) return FP8Q_ERR_UNSUPPORTED;  // one launch's
  if (work == 0) return FP8Q_OK;
  const fp8q_status o = check_overlap(tensors, count);
  if (o != FP8Q_OK) return o;
  const fp8q_status d = check_device();
  if (d != FP8Q_OK) return d;
  return launched(fp8q::launch_adamw(tensors, count, *args, grad_type == FP8Q_OUT_BF16, e4m3,
                                     stream));
}

}  // extern "C"
