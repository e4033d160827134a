// Per-token symmetric int8 quantization: BF16 rows -> int8 codes, one scale each.
//
//   s[m] = amax / 127,  q[m][k] = rne(x[m][k] * (127 * (1 / amax))),  amax = max_k |x[m][k]|
//
// (a weight matrix [N][K] gives its per-channel scales the same way).  A row is
// read once and kept in registers between its maximum and its codes, so the
// kernel moves 3 bytes an element and is bound by memory; rows too long for
// that are read a second time, from the L2.  Short rows take one wave each and
// need no LDS; longer ones 256 lanes.
//
// Arithmetic (bit-exact contract): a correctly rounded reciprocal, its rounded
// product with 127, one rounded product per element, rounding to nearest even.
// A row whose multiplier is not finite (amax 0 or below 127/FLT_MAX) is
// flushed: s = 0 and every code 0.

#include "fp8q_device.hpp"
#include "launch.hpp"

namespace fp8q {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// Elements [k, k+8) of a row of K, zeros past its end.  Rows of an odd K start
// at any even address: the load is then an unaligned one, which the memory
// system splits where it must.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t k, int64_t K) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (k + 8 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else if (k < K) {
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = k + j < K ? row[k + j] : 0u;
    v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
  }
  return v;
}

__device__ __forceinline__ float absmax8(const uint4 v) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t a = v.x & m, b = v.y & m, c = v.z & m, d = v.w & m;
  return fmaxf(fmaxf(fmaxf(bf16_lo(a), bf16_hi(a)), fmaxf(bf16_lo(b), bf16_hi(b))),
               fmaxf(fmaxf(bf16_lo(c), bf16_hi(c)), fmaxf(bf16_lo(d), bf16_hi(d))));
}

__device__ __forceinline__ uint32_t code_i8(float x, float inv) {
  const float r = rintf(x * inv);
  return (uint32_t)(int)fminf(fmaxf(r, -127.0f), 127.0f) & 0xFFu;
}

__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, float inv) {
  return code_i8(bf16_lo(a), inv) | code_i8(bf16_hi(a), inv) << 8 |
         code_i8(bf16_lo(b), inv) << 16 | code_i8(bf16_hi(b), inv) << 24;
}

// LANES lanes a row (64 or 256), V vectors of 8 elements a lane in registers;
// V = 0: any length, the row is read twice.  Kp: code row length (K up to a
// multiple of 16; the codes past K are zero).
template <int LANES, int V>
__global__ __launch_bounds__(256) void quantize_token_i8_kernel(const uint16_t* __restrict__ x,
                                                                int64_t M, int64_t K, int64_t Kp,
                                                                int8_t* __restrict__ q,
                                                                float* __restrict__ s) {
  __shared__ float red[4];
  const int t = threadIdx.x % LANES;
  const int64_t m = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (LANES == 64 && m >= M) return;  // a whole wave; with 256 lanes the grid is M
  const uint16_t* row = x + m * K;
  uint4 v[V > 0 ? V : 1];
  float a = 0.f;
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = load8(row, 8 * (int64_t)(t + LANES * i), K);
#pragma unroll
    for (int i = 0; i < V; ++i) a = fmaxf(a, absmax8(v[i]));
  } else {
    for (int64_t k = 8 * t; k < Kp; k += 8 * LANES) a = fmaxf(a, absmax8(load8(row, k, K)));
  }
  a = row16_max(a);
  a = fmaxf(a, __shfl_xor(a, 16));
  a = fmaxf(a, __shfl_xor(a, 32));
  if constexpr (LANES == 256) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
    __syncthreads();
    a = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  }
  const float inv0 = 127.0f * (1.0f / a);
  const bool flushed = !__builtin_isfinite(inv0);
  const float inv = flushed ? 0.0f : inv0;
  if (t == 0) s[m] = flushed ? 0.0f : a / 127.0f;
  int8_t* out = q + m * Kp;
  auto write = [&](int64_t k, const uint4& w) {
    if (k < Kp)
      __builtin_nontemporal_store(v2u{codes4(w.x, w.y, inv), codes4(w.z, w.w, inv)},
                                  reinterpret_cast<v2u*>(out + k));
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) write(8 * (int64_t)(t + LANES * i), v[i]);
  } else {
    for (int64_t k = 8 * t; k < Kp; k += 8 * LANES) write(k, load8(row, k, K));
  }
}

hipError_t launch_quantize_token_i8(const void* x, int64_t M, int64_t K, int64_t Kp, int8_t* q,
                                    float* s, hipStream_t stream) {
  const int rows = K <= 2048 ? 4 : 1;  // of a workgroup
  auto kern = K <= 512      ? quantize_token_i8_kernel<64, 1>
              : K <= 1024   ? quantize_token_i8_kernel<64, 2>
              : K <= 2048   ? quantize_token_i8_kernel<64, 4>
              : K <= 4096   ? quantize_token_i8_kernel<256, 2>
              : K <= 8192   ? quantize_token_i8_kernel<256, 4>
              : K <= 16384  ? quantize_token_i8_kernel<256, 8>
                            : quantize_token_i8_kernel<256, 0>;
  const int64_t slice = rows * max_blocks(256);
  for (int64_t r = 0; r < M; r += slice) {
    const int64_t n = M - r < slice ? M - r : slice;
    hipLaunchKernelGGL(kern, dim3((unsigned)((n + rows - 1) / rows)), dim3(256), 0, stream,
                       static_cast<const uint16_t*>(x) + r * K, n, K, Kp, q + r * Kp, s + r);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp8q
