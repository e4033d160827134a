// The gated block h = act(gate) * up on block-scaled E4M3 operands, in output
// tiles: the GEMM tile of gemm_tile.hpp with each wave's weight rows split into
// gate rows and the matching up rows, dense and by expert.
//
// The main loop is the GEMM's (one more multiplier per activation block and
// chunk: gate and up rows lie in two weight blocks).  What the fused epilogue
// saves is the 2F sums of a token written and read again, 8 bytes a sum in
// FP32, and a launch: at 4096 tokens, F = 2048, that is 134 MB, 27 us at the
// rate of a large copy.  There, K = 7168: 101 us, 2.38 PFLOP/s (fp8q_gemm with
// its 67 MB of FP32 results takes 115), 108 with Y saved; bound as the GEMM is,
// by the promotion and the fragment reads beside the matrix core.  By expert
// the weights' bytes bound it: 32 experts, 4300 rows 206 to 211 us, 973 MB.

#include "grouped_gemm.hpp"
#include "launch.hpp"
#include "tile_choice.hpp"

namespace fp8q {

// 256 x 256: the dense GEMM's tile.  The others are for batches that have too
// few of it to fill the CUs; their third stage is worth 46 -> 31 us at 512 rows
// (128 x 128, with 8 waves for 4), beside the second workgroup on a CU that it
// takes the room of.
using Gated256 = GemmCfg<256, 256, 4, 2, 2, 256, 1, kOpFp8, 0, 0, 1>;
using Gated256x128 = GemmCfg<256, 128, 4, 2, 3, 256, 0, kOpFp8, 0, 0, 1>;
using Gated128 = GemmCfg<128, 128, 2, 4, 3, 128, 0, kOpFp8, 0, 0, 1>;
using Gated64 = GemmCfg<64, 128, 1, 4, 3, 64, 0, kOpFp8, 0, 0, 1>;

template <class Cfg>
__global__ __launch_bounds__(Cfg::THREADS) void gated_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ SA, const uint8_t* __restrict__ W,
    const float* __restrict__ SW, int64_t M, int64_t F, int64_t K, void* __restrict__ H,
    int out_bf16, uint16_t* __restrict__ gu, int act, int tiles_n) {
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
  t.w_row0 = (int64_t)tn * (Cfg::BN / 2);
  t.w_rows = F;
  t.K = K;
  t.sa_ld = M;
  t.sw_ld = F;
  t.C = H;
  t.ldc = F;
  t.out_bf16 = out_bf16;
  t.gu = gu;
  t.act = act;
  gemm_tile<Cfg>(t, smem);
}

template <class Cfg>
static hipError_t launch_gated(const uint8_t* a_q, const float* a_s, int64_t M, const uint8_t* w_q,
                               const float* w_s, int64_t F, int64_t K, int act, void* h,
                               int out_bf16, void* gu, hipStream_t stream) {
  const int64_t tiles_n = F / (Cfg::BN / 2), tiles = (M + Cfg::BM - 1) / Cfg::BM * tiles_n;
  if (tiles > max_blocks(Cfg::THREADS)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(gated_kernel<Cfg>, dim3((unsigned)tiles), dim3(Cfg::THREADS), 0, stream, a_q,
                     a_s, w_q, w_s, M, F, K, h, out_bf16, static_cast<uint16_t*>(gu), act,
                     (int)tiles_n);
  return hipGetLastError();
}

hipError_t launch_gated_tiles(const uint8_t* a_q, const float* a_s, int64_t M, const uint8_t* w_q,
                              const float* w_s, int64_t F, int64_t K, int act, void* h,
                              int out_bf16, void* gu, int tile, hipStream_t stream) {
  auto launch = tile == tile_id(256, 256)   ? launch_gated<Gated256>
                : tile == tile_id(256, 128) ? launch_gated<Gated256x128>
                : tile == tile_id(128, 128) ? launch_gated<Gated128>
                                            : launch_gated<Gated64>;
  return launch(a_q, a_s, M, w_q, w_s, F, K, act, h, out_bf16, gu, stream);
}

#ifdef FP8Q_DEBUG_CHECKS
hipError_t gated_offsets_error_take(hipStream_t stream, int* flag) {
  return take_offsets_error(stream, flag);
}
#endif

hipError_t launch_grouped_gated_tiles(const uint8_t* a_q, const float* a_s, int64_t M_total,
                                      const int32_t* off, int G, const uint8_t* w_q,
                                      const float* w_s, int64_t F, int64_t K, int act, void* h,
                                      int out_bf16, void* gu, int cus, hipStream_t stream) {
  if (G > kMaxExpertsLds) return hipErrorInvalidValue;
  const int64_t tiles_n = (F + kGroupedBN / 2 - 1) / (kGroupedBN / 2);
  // the grid of the grouped GEMM: one workgroup for each CU, and enough of
  // them that none walks more than 64 rounds (see launch_grouped)
  const int64_t tiles = (M_total / 256 + G) * tiles_n;
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  const int64_t per_xcd = (tiles + kXcds - 1) / kXcds;
  int64_t k8 = (cus + kXcds - 1) / kXcds;
  if (k8 < (per_xcd + 63) / 64) k8 = (per_xcd + 63) / 64;
  hipLaunchKernelGGL((grouped_gemm_kernel<0, kOpFp8, 1>), dim3((unsigned)(k8 * kXcds)),
                     dim3(kGroupedThreads), 0, stream, a_q, a_s, M_total, off, G, w_q, w_s, F, K, h,
                     out_bf16, (int)tiles_n, 4 * cus, static_cast<uint16_t*>(gu), act);
  return hipGetLastError();
}

hipError_t launch_gated_few(const uint8_t* a_q, const float* a_s, int64_t M, const uint8_t* w_q,
                            const float* w_s, int64_t F, int64_t K, int act, void* h, int out_bf16,
                            void* gu, hipStream_t stream);

// off NULL: one dense block of weights; else G experts.
hipError_t launch_gemm_gated(const uint8_t* a_q, const float* a_s, int64_t M, const int32_t* off,
                             int G, const uint8_t* w_q, const float* w_s, int64_t F, int64_t K,
                             int act, void* h, int out_bf16, void* gu, hipStream_t stream) {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return hipGetLastError();
  if (off)
    return launch_grouped_gated_tiles(a_q, a_s, M, off, G, w_q, w_s, F, K, act, h, out_bf16, gu,
                                      cus, stream);
  const int tile = pick_gated(M, 2 * F, K, cus);
  if (tile == 0)
    return launch_gated_few(a_q, a_s, M, w_q, w_s, F, K, act, h, out_bf16, gu, stream);
  return launch_gated_tiles(a_q, a_s, M, w_q, w_s, F, K, act, h, out_bf16, gu, tile, stream);
}

}  // namespace fp8q
