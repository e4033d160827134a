// Block-scaled FP8 GEMM: the dense configurations and the launches of the dense
// and grouped calls.  The tile itself is in gemm_tile.hpp, the grouped kernel in
// grouped_gemm.hpp.

#include "grouped_gemm.hpp"

namespace fp8q {

// Dense configuration: 256 x 256 tiles, 8 waves (two per SIMD, so one wave's
// promotion FMAs overlap the other's MFMAs), 2 stages (132 KiB of LDS) and an
// L2 prefetch kPfDist chunks ahead (a ring of 2 stages leaves the loads of a
// chunk less than one chunk's compute time to arrive from HBM).
using DenseCfg = GemmCfg<256, 256, 4, 2, 2, 256, 1>;
// The BF16 GEMM: the same tile, waves, ring and prefetch.
using DenseBf16Cfg = GemmCfg<256, 256, 4, 2, 2, 256, 1, kOpBf16>;
// The precise mode: the same tile, waves, ring and prefetch, FP16 MFMAs on
// the widened codes.
using DenseWideCfg = GemmCfg<256, 256, 4, 2, 2, 256, 1, kOpWide16>;
// Power-of-two scales applied by the matrix core: the same tile, waves, ring
// and prefetch.
using DenseMxCfg = GemmCfg<256, 256, 4, 2, 2, 256, 1, kOpFp8Mx>;
// The weight-gradient GEMM: the dense tile with row-scaled weights.
using RowScaledCfg = GemmCfg<256, 256, 4, 2, 2, 256, 1, kOpFp8, 1>;
using RowScaledWideCfg = GemmCfg<256, 256, 4, 2, 2, 256, 1, kOpWide16, 1>;
// The same with 224-row weight tiles (waves of 64 x 112; row-scaled weights
// have no 128-row blocks to respect), for shapes where they fill the CUs'
// rounds better: 4096 x 7168 outputs make 448 tiles of 256 x 256 (a second
// round 3/4 full on 256 CUs) but 512 of 256 x 224 (two full rounds of
// 7/8-size tiles).  No L2 prefetch (its share is laid out for 256 x 256).
using RowScaled224Cfg = GemmCfg<256, 224, 4, 2, 2, 256, 0, kOpFp8, 1>;
// BF16 activations quantized inside the GEMM (scale mode MODE): the dense
// tile without the L2 prefetch, whose A lines would be BF16 rows.
template <int MODE>
using DenseCastCfg = GemmCfg<256, 256, 4, 2, 2, 256, 0, kOpFp8, 0, 1 + MODE>;
template <class Cfg>
__global__ __launch_bounds__(Cfg::THREADS) void gemm_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ SA, const uint8_t* __restrict__ W,
    const float* __restrict__ SW, int64_t M, int64_t N, int64_t K, void* __restrict__ C,
    int out_bf16, int tiles_n) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[Cfg::LDS_BYTES];
  int tm, tn;
  xcd_tile(blockIdx.x, gridDim.x, tiles_n, tm, tn);
  TileArgs t;
  t.A = A;
  t.SA = SA;
  t.W = W;
  t.SW = SW;
  t.a_row0 = (int64_t)tm * Cfg::BM;
  t.a_rows = M;
  t.w_row0 = (int64_t)tn * Cfg::BN;
  t.w_rows = N;
  t.K = K;
  t.sa_ld = M;
  t.sw_ld = N;
  t.C = C;
  t.ldc = N;
  t.out_bf16 = out_bf16;
  t.gu = nullptr;
  t.act = 0;
  gemm_tile<Cfg>(t, smem);
}

#ifdef FP8Q_DEBUG_CHECKS
hipError_t offsets_error_take(hipStream_t stream, int* flag) {
  return take_offsets_error(stream, flag);
}
#endif

hipError_t launch_gemm_bf16(const void* a, const void* w, int64_t M, int64_t N, int64_t K,
                            void* c, int out_bf16, hipStream_t stream) {
  using Cfg = DenseBf16Cfg;
  if (M == 0 || N == 0) return hipSuccess;
  const int64_t tiles_m = (M + Cfg::BM - 1) / Cfg::BM;
  const int64_t tiles_n = (N + Cfg::BN - 1) / Cfg::BN;
  const int64_t tiles = tiles_m * tiles_n;
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  // Operand rows are 2K bytes: the kernel's K is the row length in bytes.
  hipLaunchKernelGGL(gemm_kernel<Cfg>, dim3((unsigned)tiles), dim3(Cfg::THREADS), 0, stream,
                     static_cast<const uint8_t*>(a), nullptr, static_cast<const uint8_t*>(w),
                     nullptr, M, N, 2 * K, c, out_bf16, (int)tiles_n);
  return hipGetLastError();
}

template <class Cfg>
static hipError_t launch_rowscaled_cfg(const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                                       const float* b_s, int64_t M, int64_t N, int64_t K, void* c,
                                       int out_bf16, hipStream_t stream) {
  const int64_t tiles_m = (M + Cfg::BM - 1) / Cfg::BM;
  const int64_t tiles_n = (N + Cfg::BN - 1) / Cfg::BN;
  const int64_t tiles = tiles_m * tiles_n;
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL(gemm_kernel<Cfg>, dim3((unsigned)tiles), dim3(Cfg::THREADS), 0, stream, a_q,
                     a_s, b_q, b_s, M, N, K, c, out_bf16, (int)tiles_n);
  return hipGetLastError();
}

hipError_t launch_gemm_rowscaled(const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                                 const float* b_s, int64_t M, int64_t N, int64_t K, void* c,
                                 int out_bf16, int precise, hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  if (precise)
    return launch_rowscaled_cfg<RowScaledWideCfg>(a_q, a_s, b_q, b_s, M, N, K, c, out_bf16,
                                                  stream);
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return hipGetLastError();
  // Rounds of tiles over the CUs times the tile width: the 224-row weight
  // tiles when they finish sooner by that measure.
  const int64_t tm = (M + 255) / 256;
  const int64_t r256 = (tm * ((N + 255) / 256) + cus - 1) / cus;
  const int64_t r224 = (tm * ((N + 223) / 224) + cus - 1) / cus;
  if (r224 * 224 < r256 * 256)
    return launch_rowscaled_cfg<RowScaled224Cfg>(a_q, a_s, b_q, b_s, M, N, K, c, out_bf16, stream);
  return launch_rowscaled_cfg<RowScaledCfg>(a_q, a_s, b_q, b_s, M, N, K, c, out_bf16, stream);
}

hipError_t launch_gemm(const uint8_t* a_q, const float* a_s, const uint8_t* w_q,
                       const float* w_s, int64_t M, int64_t N, int64_t K, void* c, int out_bf16,
                       int mode, hipStream_t stream) {
  using Cfg = DenseCfg;
  static_assert(DenseWideCfg::BM == Cfg::BM && DenseWideCfg::BN == Cfg::BN, "same tiles");
  static_assert(DenseMxCfg::BM == Cfg::BM && DenseMxCfg::BN == Cfg::BN, "same tiles");
  if (M == 0 || N == 0) return hipSuccess;
  const int64_t tiles_m = (M + Cfg::BM - 1) / Cfg::BM;
  const int64_t tiles_n = (N + Cfg::BN - 1) / Cfg::BN;
  const int64_t tiles = tiles_m * tiles_n;
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  // mode 0: FP8 MFMA; 1: the precise mode; 2: scales applied by the matrix core
  auto kern = mode == 1 ? gemm_kernel<DenseWideCfg>
              : mode == 2 ? gemm_kernel<DenseMxCfg> : gemm_kernel<Cfg>;
  hipLaunchKernelGGL(kern, dim3((unsigned)tiles), dim3(Cfg::THREADS), 0, stream, a_q, a_s, w_q,
                     w_s, M, N, K, c, out_bf16, (int)tiles_n);
  return hipGetLastError();
}

// BF16 activations x quantized inside the dense GEMM (scale mode `mode`).
hipError_t launch_gemm_cast(const void* x, const uint8_t* w_q, const float* w_s, int64_t M,
                            int64_t N, int64_t K, void* c, int out_bf16, int mode,
                            hipStream_t stream) {
  using Cfg = DenseCastCfg<0>;
  static_assert(DenseCastCfg<1>::BM == Cfg::BM && DenseCastCfg<1>::BN == Cfg::BN, "same tiles");
  if (M == 0 || N == 0) return hipSuccess;
  const int64_t tiles_m = (M + Cfg::BM - 1) / Cfg::BM;
  const int64_t tiles_n = (N + Cfg::BN - 1) / Cfg::BN;
  const int64_t tiles = tiles_m * tiles_n;
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = mode == 0 ? gemm_kernel<DenseCastCfg<0>> : gemm_kernel<DenseCastCfg<1>>;
  hipLaunchKernelGGL(kern, dim3((unsigned)tiles), dim3(Cfg::THREADS), 0, stream,
                     static_cast<const uint8_t*>(x), nullptr, w_q, w_s, M, N, K, c, out_bf16,
                     (int)tiles_n);
  return hipGetLastError();
}

// cast = 0: a holds FP8 codes with scales a_s; cast = 1 + mode: a holds BF16
// activations quantized inside the kernel (a_s unused); cast = -1: FP8 codes
// through the precise mode.
static hipError_t launch_grouped(const uint8_t* a, const float* a_s, int64_t M_total,
                                 const int32_t* off, int G, const uint8_t* w_q,
                                 const float* w_s, int64_t N, int64_t K, void* c, int out_bf16,
                                 int cast, hipStream_t stream) {
  if (M_total == 0 || N == 0) return hipSuccess;
  if (G > kMaxExpertsLds) return hipErrorInvalidValue;
  const int64_t tiles_n = (N + kGroupedBN - 1) / kGroupedBN;
  // sum_e ceil(M_e / 256) <= floor(M_total / 256) + G
  const int64_t max_mtiles = M_total / 256 + G;
  const int64_t tiles = max_mtiles * tiles_n;
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return hipGetLastError();
  // Persistent grid: one workgroup per CU (LDS allows one), 8 per XCD
  // round, and enough of them that no workgroup walks more than 64 rounds of
  // its XCD's run (at most ceil(tiles / 8) tiles).
  const int64_t per_xcd = (tiles + kXcds - 1) / kXcds;
  int64_t k8 = (cus + kXcds - 1) / kXcds;
  if (k8 < (per_xcd + 63) / 64) k8 = (per_xcd + 63) / 64;
  const int64_t grid = k8 * kXcds;
  // The largest-first order applies up to 4 tiles per CU of the device.
  auto kern = cast == -1  ? grouped_gemm_kernel<0, kOpWide16>
              : cast == 0 ? grouped_gemm_kernel<0>
              : cast == 1 ? grouped_gemm_kernel<1>
                          : grouped_gemm_kernel<2>;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kGroupedThreads), 0, stream, a, a_s,
                     M_total, off, G, w_q, w_s, N, K, c, out_bf16, (int)tiles_n, 4 * cus, nullptr,
                     0);
  return hipGetLastError();
}

hipError_t launch_grouped_gemm(const uint8_t* a_q, const float* a_s, int64_t M_total,
                               const int32_t* off, int G, const uint8_t* w_q, const float* w_s,
                               int64_t N, int64_t K, void* c, int out_bf16, int precise,
                               hipStream_t stream) {
  return launch_grouped(a_q, a_s, M_total, off, G, w_q, w_s, N, K, c, out_bf16,
                        precise ? -1 : 0, stream);
}

hipError_t launch_grouped_gemm_cast(const void* x, int64_t M_total, const int32_t* off, int G,
                                    const uint8_t* w_q, const float* w_s, int64_t N, int64_t K,
                                    void* c, int out_bf16, int mode, hipStream_t stream) {
  return launch_grouped(static_cast<const uint8_t*>(x), nullptr, M_total, off, G, w_q, w_s, N,
                        K, c, out_bf16, 1 + mode, stream);
}

}  // namespace fp8q
