// Layer norm over the rows of x[M][N], and its backward pass.
//
//   z = (x - mean) rstd,  y = z weight + bias,  rstd = 1 / sqrt(var + eps);
//   gz = dy weight,  dx = rstd (gz - mean(gz) - z mean(gz z)),
//   dweight = sum over rows of dy z,  dbias = sum over rows of dy.
//
// A row stays in registers (LPR lanes, NV pieces of 8 consecutive elements each):
// it is read once, its variance is taken about its mean in a second pass over
// the registers, and y leaves as E4M3 codes (128 consecutive elements are one DPP
// row of 16 lanes, so a group's maximum costs four instructions), as BF16 or
// FP32, or both: bound by memory.  The codes are those of y in FP32, not of its
// BF16 rounding.  4096 rows of 7168, FP32 in, codes and BF16 out: 41 us over two sets of
// inputs in turn (5.0 TB/s, a copy's rate), 45 over more of them.
//
// Rows whose squares or sums leave FP32's range are read and summed again, scaled by a
// power of two; the others pay a comparison for it (under 1%).
//
// Backward: each workgroup walks rows and keeps its columns' sums of dy z and dy
// in registers; they go to a workspace, one row of it a workgroup, which a second
// kernel adds up in a fixed order (no atomics: the same bits every time).  4096 rows of
// 7168, x and dx in FP32, dy in BF16: 68 to 71 us (4.2 TB/s); what the workgroups leave,
// 15 MB that are written and read, takes 7 of them.  Five kernels for widths that are no
// multiple of 8 keep 7 to 13 registers in scratch memory: FP32 x and dy of 4097 to 8192
// columns, and all types above 8192.

#include <type_traits>

#include "activation.hpp"
#include "fp8q.h"
#include "launch.hpp"
#include "quant_rules.hpp"

namespace fp8q {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
// 16 bytes at any element's address: rows of odd N start anywhere
typedef v4u v4u_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

struct Row8 {
  float v[8];
};

// Elements 8c .. 8c+7 of a row of n as they are in memory; those past the row are 0.
// WHOLE: n is a multiple of 8, no piece ends early (the code for one that does takes
// registers, which in the backward pass are the rows under way).
template <bool BF16>
struct Raw8 {
  v4u w[BF16 ? 1 : 2];
};

template <bool BF16, bool WHOLE>
__device__ __forceinline__ Raw8<BF16> load_raw(const void* row, int c, int n) {
  Raw8<BF16> r;
  const int i = 8 * c;
  if (i + 8 <= n) {
    const char* at = static_cast<const char*>(row) + (int64_t)i * (BF16 ? 2 : 4);
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) r.w[h] = *reinterpret_cast<const v4u_any*>(at + 16 * h);
  } else if (WHOLE) {
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) r.w[h] = v4u{0, 0, 0, 0};
  } else {
    uint32_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      e[j] = 0;
      if (i + j < n)
        e[j] = BF16 ? (uint32_t)static_cast<const uint16_t*>(row)[i + j]
                    : static_cast<const uint32_t*>(row)[i + j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF16) {
        r.w[0][j] = e[2 * j] | (e[2 * j + 1] << 16);
      } else {
        r.w[0][j] = e[j];
        r.w[1][j] = e[4 + j];
      }
    }
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ Row8 widened(const Raw8<BF16>& r) {
  Row8 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (BF16) {
      o.v[2 * j] = bf16_lo(r.w[0][j]);
      o.v[2 * j + 1] = bf16_hi(r.w[0][j]);
    } else {
      o.v[j] = __uint_as_float(r.w[0][j]);
      o.v[4 + j] = __uint_as_float(r.w[1][j]);
    }
  }
  return o;
}

template <bool BF16, bool WHOLE>
__device__ __forceinline__ Row8 load8(const void* row, int c, int n) {
  return widened<BF16>(load_raw<BF16, WHOLE>(row, c, n));
}

template <bool BF16, bool WHOLE>
__device__ __forceinline__ void store8(void* row, int c, int n, const Row8& r) {
  const int i = 8 * c;
  if (WHOLE || i + 8 <= n) {  // (the caller's pieces begin within the row)
    if constexpr (BF16) {
      v4u w;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack_bf16x2(r.v[2 * j], r.v[2 * j + 1]);
      *reinterpret_cast<v4u_any*>(static_cast<uint16_t*>(row) + i) = w;
    } else {
      *reinterpret_cast<v4f_any*>(static_cast<float*>(row) + i) =
          v4f{r.v[0], r.v[1], r.v[2], r.v[3]};
      *reinterpret_cast<v4f_any*>(static_cast<float*>(row) + i + 4) =
          v4f{r.v[4], r.v[5], r.v[6], r.v[7]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) {
        if constexpr (BF16)
          static_cast<uint16_t*>(row)[i + j] = (uint16_t)pack_bf16x2(r.v[j], 0.f);
        else
          static_cast<float*>(row)[i + j] = r.v[j];
      }
  }
}

template <class T>
__device__ __forceinline__ T* row_at(T* base, int64_t row, int64_t n, bool bf16) {
  return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(base) + row * n * (bf16 ? 2 : 4));
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}

// Sum over 16, 32 or 64 lanes of the wave, the same in every lane of them: over DPP
// rows of 16 in the vector ALU (each step adds a lane's mirror image, so both have the
// same sum), then the rows'.  (Through LDS, as a shuffle goes, each step waits for it.)
template <int LANES>
__device__ __forceinline__ float lane_sum(float v) {
  v = dpp_add<kDppQuadXor1>(v);
  v = dpp_add<kDppQuadXor2>(v);
  v = dpp_add<kDppRowHalfMirror>(v);
  v = dpp_add<kDppRowMirror>(v);
  if constexpr (LANES == 16) return v;
  auto row = [&](int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
  };
  const float lo = row(0) + row(16), hi = row(32) + row(48);
  if constexpr (LANES == 32) return (threadIdx.x & 32) ? hi : lo;
  return lo + hi;
}

// Sums of K values over the LPR lanes of a row; every lane gets them.  `red`
// holds K values of each wave; calls alternate between two such places.
template <int LPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*red)[16]) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane_sum<LPR < 64 ? LPR : 64>(v[k]);
  if constexpr (LPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) red[k][wave] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v4f s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < LPR / 64; w += 4) s += *reinterpret_cast<const v4f*>(&red[k][w]);
      v[k] = (s[0] + s[1]) + (s[2] + s[3]);
    }
  }
}

struct NormArgs {
  const void* x;
  const float* weight;
  const float* bias;
  int64_t M;
  int N;
  float eps;
  void* y;
  int y_bf16;
  uint8_t* q;
  float* s;
  int mode;
  float* mean;
  float* rstd;
};

constexpr int kCus = 256;

// Variances (and eps) from here up have lost nothing: a square below FP32's normals is
// off by 2^-150.
constexpr float kLeastVar = 0x1p-96f, kMost = 0x1.fffffep127f;

template <int LPR>
constexpr int kRowThreads = LPR < 256 ? 256 : LPR;

template <int MODE>
__device__ __forceinline__ void store_codes(const NormArgs& a, int64_t row, int c, const Row8& y) {
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y.v[j]));
  const GroupRule r = group_rule<MODE>(row16_max(amax));
  const v2u o = {pack_e4m3x4(apply<MODE>(y.v[0], r), apply<MODE>(y.v[1], r), apply<MODE>(y.v[2], r),
                             apply<MODE>(y.v[3], r)),
                 pack_e4m3x4(apply<MODE>(y.v[4], r), apply<MODE>(y.v[5], r), apply<MODE>(y.v[6], r),
                             apply<MODE>(y.v[7], r))};
  *reinterpret_cast<v2u*>(a.q + row * a.N + 8 * c) = o;
  if ((threadIdx.x & 15) == 0) a.s[(int64_t)(c >> 4) * a.M + row] = r.s;
}

template <bool X_BF16, int LPR, int NV, bool WHOLE>
__global__ __launch_bounds__(kRowThreads<LPR>) void layer_norm_kernel(const NormArgs a) {
  __shared__ __attribute__((aligned(16))) float red[2][1][16];
  constexpr int RPW = kRowThreads<LPR> / LPR;
  const int l = threadIdx.x % LPR;
  const int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / LPR;
  if (RPW > 1 && row >= a.M) return;  // (whole DPP rows, and no barrier follows)
  const int N = a.N;
  const void* x = row_at(a.x, row, N, X_BF16);
  Row8 v[NV];
  float sum[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    v[j] = load8<X_BF16, WHOLE>(x, l + LPR * j, N);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[0] += v[j].v[k];
  }
  row_sum<LPR, 1>(sum, red[0]);
  float mean = sum[0] / (float)N;
  float sq[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = 8 * (l + LPR * j) + k < N ? v[j].v[k] - mean : 0.f;
      v[j].v[k] = d;
      sq[0] = __builtin_fmaf(d, d, sq[0]);
    }
  row_sum<LPR, 1>(sq, red[1]);
  float var = sq[0] / (float)N + a.eps, scale = 1.f;
  if (!(var >= kLeastVar && var <= kMost)) {
    // Rare, and the same for all lanes of a row: sums that overflow or squares that
    // underflow.  The row again, large values times 2^-100 or small deviations times
    // 2^100 (the largest sum of squares is then 2^70, the least square 2^-98).
    const bool small = var < kLeastVar;
    const float before = small ? 1.f : 0x1p-100f, after = small ? 0x1p100f : 1.f;
    sum[0] = sq[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      v[j] = load8<X_BF16, WHOLE>(x, l + LPR * j, N);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[0] += v[j].v[k] *= before;
    }
    row_sum<LPR, 1>(sum, red[0]);
    const float m = sum[0] / (float)N;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = 8 * (l + LPR * j) + k < N ? (v[j].v[k] - m) * after : 0.f;
        v[j].v[k] = d;
        sq[0] = __builtin_fmaf(d, d, sq[0]);
      }
    row_sum<LPR, 1>(sq, red[1]);
    scale = sq[0] == 0.f ? 1.f : before * after;  // (of a constant row eps alone is left)
    mean = small ? m : m * 0x1p100f;
    var = sq[0] / (float)N + a.eps * scale * scale;
  }
  const float rstd = 1.f / __builtin_sqrtf(var);  // of the deviations in v
  if (l == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd * scale;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = l + LPR * j;
    if (8 * c >= N) continue;
    const Row8 w = load8<false, WHOLE>(a.weight, c, N);
    Row8 y;
    if (a.bias) {
      const Row8 b = load8<false, WHOLE>(a.bias, c, N);
#pragma unroll
      for (int k = 0; k < 8; ++k) y.v[k] = __builtin_fmaf(v[j].v[k] * rstd, w.v[k], b.v[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) y.v[k] = v[j].v[k] * rstd * w.v[k];
    }
    if (a.q) {
      if (a.mode == 0)
        store_codes<0>(a, row, c, y);
      else
        store_codes<1>(a, row, c, y);
    }
    if (a.y) {
      if (a.y_bf16)
        store8<true, WHOLE>(row_at(a.y, row, N, true), c, N, y);
      else
        store8<false, WHOLE>(row_at(a.y, row, N, false), c, N, y);
    }
  }
}

// ------------------------------------------------------------------ backward
struct NormBwArgs {
  const void* dy;
  const void* x;
  const float* weight;
  const float* mean;
  const float* rstd;
  int64_t M;
  int N;
  void* dx;
  float* dw;        // of workgroup b: dw + b * stride, db + b * stride
  float* db;        // (one workgroup: the results themselves; db may then be NULL)
  int64_t stride;
};

template <bool X_BF16, bool DY_BF16, int LPR, int NV, bool WHOLE>
__global__ __launch_bounds__(kRowThreads<LPR>) void layer_norm_backward_kernel(const NormBwArgs a) {
  __shared__ __attribute__((aligned(16))) float red[2][2][16];
  constexpr int RPW = kRowThreads<LPR> / LPR;
  const int l = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int N = a.N;
  const float inv_n = 1.f / (float)N;
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[j][k] = db[j][k] = 0.f;
  const int64_t step = (int64_t)gridDim.x * RPW;
  int64_t row = (int64_t)blockIdx.x * RPW + sub;
  // The next two rows' values are on their way while one is worked on (of the widest
  // rows there are no registers for them).
  constexpr bool kAhead = LPR * NV < 2048;
  struct Values {
    Raw8<X_BF16> x[NV];
    Raw8<DY_BF16> dy[NV];
    float mean, rstd;
  };
  auto load = [&](Values& v, int64_t r) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      v.x[j] = load_raw<X_BF16, WHOLE>(row_at(a.x, r, N, X_BF16), l + LPR * j, N);
      v.dy[j] = load_raw<DY_BF16, WHOLE>(row_at(a.dy, r, N, DY_BF16), l + LPR * j, N);
    }
    v.mean = a.mean[r];
    v.rstd = a.rstd[r];
  };
  // Row `row`, whose values are in v, which then takes those of the row after the next.
  auto one = [&](Values& v, float (*red)[16]) {
    const float mean = v.mean, rstd = v.rstd;
    Row8 z[NV], g[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      z[j] = widened<X_BF16>(v.x[j]);
      g[j] = widened<DY_BF16>(v.dy[j]);
    }
    if (kAhead && row + 2 * step < a.M) load(v, row + 2 * step);
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Row8 w = load8<false, WHOLE>(a.weight, l + LPR * j, N);
      // (past the row z is 0 as well: a mean times rstd that overflows would make its
      // product with dy's 0 a NaN)
      const float m = !WHOLE || 8 * (l + LPR * j) < N ? mean : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = WHOLE || 8 * (l + LPR * j) + k < N ? z[j].v[k] - m : 0.f;
        const float zz = d * rstd;
        z[j].v[k] = zz;
        dw[j][k] = __builtin_fmaf(g[j].v[k], zz, dw[j][k]);
        db[j][k] += g[j].v[k];
        g[j].v[k] *= w.v[k];
        sum[0] += g[j].v[k];
        sum[1] = __builtin_fmaf(g[j].v[k], zz, sum[1]);
      }
    }
    row_sum<LPR, 2>(sum, red);
    const float c2 = sum[0] * inv_n, c1 = sum[1] * inv_n;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = l + LPR * j;
      Row8 d;
#pragma unroll
      for (int k = 0; k < 8; ++k) d.v[k] = rstd * (g[j].v[k] - c2 - z[j].v[k] * c1);
      if (8 * c < N) store8<X_BF16, WHOLE>(row_at(a.dx, row, N, X_BF16), c, N, d);
    }
    row += step;
  };
  Values v0, v1;
  if (kAhead) {
    if (row < a.M) load(v0, row);
    if (row + step < a.M) load(v1, row + step);
  }
  while (row < a.M) {
    if (!kAhead) load(v0, row);
    one(v0, red[0]);
    if (row >= a.M) break;
    if (!kAhead) load(v1, row);
    one(v1, red[1]);
  }
  if constexpr (RPW > 1) {
    // the lane groups' sums of the same columns, one group after the other
    __shared__ float part[2][RPW][NV][8][LPR];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        part[0][sub][j][k][l] = dw[j][k];
        part[1][sub][j][k][l] = db[j][k];
      }
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        for (int s = 1; s < RPW; ++s) {
          dw[j][k] += part[0][s][j][k][l];
          db[j][k] += part[1][s][j][k][l];
        }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = l + LPR * j;
    Row8 w, b;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      w.v[k] = dw[j][k];
      b.v[k] = db[j][k];
    }
    if (8 * c < N) {
      store8<false, WHOLE>(a.dw + blockIdx.x * a.stride, c, N, w);
      if (a.db) store8<false, WHOLE>(a.db + blockIdx.x * a.stride, c, N, b);
    }
  }
}

// Column sums of part[rows][2N]: 32 columns x 32 slices of the rows a workgroup.
__global__ __launch_bounds__(1024) void layer_norm_reduce_kernel(const float* __restrict__ part,
                                                                 int rows, int N,
                                                                 float* __restrict__ dweight,
                                                                 float* __restrict__ dbias) {
  __shared__ float red[32][33];
  const int l = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t ld = 2 * (int64_t)N, col = (int64_t)blockIdx.x * 32 + l;
  float s = 0.f;
  if (col < ld) {
    // slice, slice + 32, ...: the rows that are loaded together follow each other
#pragma unroll 4
    for (int r = slice; r < rows; r += 32) s += part[r * ld + col];
  }
  red[slice][l] = s;
  __syncthreads();
  // lane i of a wave's half adds up column `slice`
  s = red[l][slice];
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor(s, d);
  const int64_t out = (int64_t)blockIdx.x * 32 + slice;
  if (l != 0 || out >= ld) return;
  if (out < N)
    dweight[out] = s;
  else if (dbias)
    dbias[out - N] = s;
}

// ------------------------------------------------------------------ launches
// Lanes of a row and pieces of a lane that fit the row, for both passes.  Four or two
// narrow rows share a wave (200000 rows of 128: 19 us, a wave each 58; backward, 100000
// rows: 20.6 and 37).  The wide rows of the forward pass take two pieces a lane (4096
// rows of 7168: 42 us, one piece 48); those of the backward pass one, which leaves
// registers for the rows under way.
template <int LPR, int NV>
struct Width {
  static constexpr int kLpr = LPR, kNv = NV;
};

template <bool BACKWARD, class F>
static hipError_t by_width(int64_t N, F f) {
  const int64_t c = (N + 7) / 8;
  auto g = [&](auto w) {
    return N % 8 == 0 ? f(w, std::true_type{}) : f(w, std::false_type{});
  };
  if (c <= 16) return g(Width<16, 1>{});
  if (c <= 32) return g(Width<32, 1>{});
  if (c <= 64) return g(Width<64, 1>{});
  if (c <= 128) return g(Width<64, 2>{});
  if (c <= 256) return g(Width<256, 1>{});
  if constexpr (BACKWARD) {
    if (c <= 512) return g(Width<512, 1>{});
    if (c <= 1024) return g(Width<1024, 1>{});
  } else {
    if (c <= 512) return g(Width<256, 2>{});
    if (c <= 1024) return g(Width<512, 2>{});
  }
  return g(Width<1024, 2>{});
}

hipError_t launch_layer_norm(const void* x, int x_bf16, const float* weight, const float* bias,
                             int64_t M, int64_t N, float eps, void* y, int y_bf16, uint8_t* q,
                             float* s, int mode, float* mean, float* rstd, hipStream_t stream) {
  const NormArgs a = {x, weight, bias, M, (int)N, eps, y, y_bf16, q, s, mode, mean, rstd};
  return by_width<false>(N, [&](auto w, auto whole) {
    constexpr int LPR = decltype(w)::kLpr, NV = decltype(w)::kNv, T = kRowThreads<LPR>;
    constexpr bool WHOLE = decltype(whole)::value;
    const int64_t blocks = (M + T / LPR - 1) / (T / LPR);
    if (blocks > max_blocks(T)) return hipErrorInvalidValue;
    auto kern = x_bf16 ? layer_norm_kernel<true, LPR, NV, WHOLE>
                       : layer_norm_kernel<false, LPR, NV, WHOLE>;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(T), 0, stream, a);
    return hipGetLastError();
  });
}

// Workgroups of the backward pass.  One for a few rows (it writes the results
// itself); else enough to fill the chip, but with kRowsEach rows for each lane group
// at least, so that what the workgroups leave to be added up stays small.
// (4096 rows of 7168 in 256 workgroups of 1024 lanes: 70.7 us, in 512 78.5.)
constexpr int kNormThreads = 1024 * 256, kRowsEach = 8, kRowsAlone = 2;

static int64_t norm_backward_blocks(int64_t M, int64_t N) {
  int64_t blocks = 0;
  (void)by_width<true>(N, [&](auto w, auto) {
    constexpr int LPR = decltype(w)::kLpr, T = kRowThreads<LPR>, RPW = T / LPR;
    const int64_t rows = (M + RPW - 1) / RPW, most = kNormThreads / T;
    blocks = (rows + kRowsEach - 1) / kRowsEach;
    blocks = blocks > most ? most : blocks;
    const int64_t least = rows < kCus ? rows : kCus;
    blocks = rows <= kRowsAlone ? 1 : blocks < least ? least : blocks;
    return hipSuccess;
  });
  return M == 0 ? 0 : blocks;
}

int64_t layer_norm_backward_workspace(int64_t M, int64_t N) {
  const int64_t blocks = norm_backward_blocks(M, N);
  return blocks > 1 ? blocks * 2 * N * 4 : 0;
}

hipError_t launch_layer_norm_backward(const void* dy, int dy_bf16, const void* x, int x_bf16,
                                      const float* weight, const float* mean, const float* rstd,
                                      int64_t M, int64_t N, void* dx, float* dweight, float* dbias,
                                      float* workspace, hipStream_t stream) {
  const int blocks = (int)norm_backward_blocks(M, N);
  NormBwArgs a = {dy, x, weight, mean, rstd, M, (int)N, dx, workspace, workspace + N, 2 * N};
  if (blocks == 1) {
    a.dw = dweight;
    a.db = dbias;
  }
  const hipError_t e = blocks == 0 ? hipSuccess : by_width<true>(N, [&](auto w, auto whole) {
    constexpr int LPR = decltype(w)::kLpr, NV = decltype(w)::kNv;
    constexpr bool WHOLE = decltype(whole)::value;
    auto kern = x_bf16 ? (dy_bf16 ? layer_norm_backward_kernel<true, true, LPR, NV, WHOLE>
                                  : layer_norm_backward_kernel<true, false, LPR, NV, WHOLE>)
                       : (dy_bf16 ? layer_norm_backward_kernel<false, true, LPR, NV, WHOLE>
                                  : layer_norm_backward_kernel<false, false, LPR, NV, WHOLE>);
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kRowThreads<LPR>), 0, stream, a);
    return hipGetLastError();
  });
  if (e != hipSuccess || blocks == 1) return e;
  hipLaunchKernelGGL(layer_norm_reduce_kernel, dim3((unsigned)((2 * N + 31) / 32)), dim3(1024), 0,
                     stream, workspace, blocks, (int)N, dweight, dbias);
  return hipGetLastError();
}

}  // namespace fp8q
