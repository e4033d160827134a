// Block-scaled FP8 GEMM with FP32 promotion every 128 K, dense and grouped.
//
// Method: why-be.co.kr as_center post 57820, promotion passage (at the end of
// every N_C interval the partial result leaves the matrix unit, is multiplied
// by the scaling factors and added into FP32 registers on the general ALUs);
// pkd.ac.th webboard post 78017, increased-precision accumulation passage
// (N_C = 128); the-good.kr free board post 2169793 (per-group scaling along K,
// dequantized on the general ALUs).
//
// MI355X mapping.  One v_mfma_f32_16x16x128_f8f6f4 consumes exactly one
// 128-wide K chunk of a 16x16 output block, so each chunk's partial P_g is a
// single MFMA started from zero; the promotion acc = fma(P_g, s_a*s_w, acc) is
// four VALU FMAs per MFMA.  The product is formed transposed (C^T = W A^T:
// MFMA rows are weight rows, MFMA columns are activation rows), so a lane's
// four results of a block share one activation row and one multiplier, and
// are four consecutive outputs (one 16-byte store).  Inside a wave the blocks
// are software pipelined: block k's partial is folded by the VALU while the
// matrix core runs the next MFMAs (the role the pages give to two alternating
// warpgroups on Hopper).
//
// Each wave owns 64 (48 in the grouped 160- and 192-row tiles) activation rows
// and 128 weight rows inside one 128-row weight block, so s_w is one
// wave-uniform scalar per chunk, and the row scales of a row of waves are one
// 256-byte LDS slot per chunk.  Operands move HBM/L2 -> LDS with 16-byte
// direct-to-LDS buffer loads (no VGPR staging) through a ring of STAGES K
// chunks with one barrier per chunk; the loads of the chunks ahead are spread
// over the MFMA sequence, and the next chunk's fragments are read
// into registers before the current chunk's last MFMAs, so the matrix core
// does not drain at chunk boundaries.  LDS rows are 128 bytes (one K chunk)
// with the 16-byte column index XOR-swizzled per row so fragment reads are
// bank-conflict free.  The dense kernel's two-stage ring is backed by an L2
// prefetch several chunks ahead, split between the tiles that share a band
// of A or W rows in one XCD's L2.
//
// The same tile serves more configurations (GemmCfg flags): the
// weight-gradient GEMM, whose weight-side operand carries 1x128 row-group
// scales like the activations (W_ROWSCALE: the multiplier differs per output
// element); BF16 operands without scales (OP = kOpBf16: the reference of the
// FP8 path, accumulating in the matrix core); the precise mode (OP =
// kOpWide16: the E4M3 codes, unchanged in LDS, are widened exactly to FP16 in
// registers and each chunk's partial is formed by FP16 MFMAs, whose FP32
// accumulation has no narrow truncation step); power-of-two scales applied by
// the matrix core as E8M0 operand scales (OP = kOpFp8Mx, the pages' "MMA with
// group scaling" wish: the partial comes out scaled and the promotion is an
// add); BF16 activations quantized on their way into LDS (A_CAST, see
// ACaster); the gated block act(gate) * up (GATED: each wave's weight rows are
// gate rows and the matching up rows, so that a lane holds both sums of an
// output and the epilogue needs no exchange); and the grouped MoE kernel's
// row-count buckets (persistent workgroups, see grouped_gemm_kernel).

#pragma once

#include <type_traits>

#include "activation.hpp"
#include "gemm_common.hpp"
#include "quant_rules.hpp"

namespace fp8q {

// OP_: the operands and the matrix-core instruction.
//   kOpFp8   : E4M3 codes; one 16x16x128 FP8 MFMA forms a block's chunk
//              partial from zero.
//   kOpBf16  : BF16 operands (the reference GEMM of the same kernel family):
//              a 128-byte stage row then holds 64 K values, each 16x16 block
//              takes two chained 16x16x32 BF16 MFMAs per chunk, accumulating
//              in the matrix core (its BF16 path accumulates to FP32
//              accuracy), and there are no scales.
//   kOpWide16: E4M3 codes staged exactly as for kOpFp8, widened to FP16 in
//              registers after the fragment read (exact: every E4M3 value is
//              an FP16 value), and a block's chunk partial is four chained
//              16x16x32 FP16 MFMAs from zero (the precise mode: the FP8
//              MFMA truncates products inside 8-product groups, the FP16 one
//              accumulates its exact products to FP32 accuracy).
//   kOpFp8Mx : E4M3 codes with power-of-two scales, which the matrix core
//              applies itself: the block-scaled FP8 MFMA takes each group
//              scale as an E8M0 byte (the lanes that supply a row's operand
//              supply its byte), so a chunk partial comes out already
//              scaled, from zero, and the promotion is a plain FP32 add.
// W_ROWSCALE_: the weight-side operand carries 1x128 row-group scales
// ([K/128][N], like the activations) instead of 128x128 block scales: the
// weight-gradient GEMM, whose operands dY^T and X^T are both grouped along
// the tokens.  The multiplier then differs per output element.
// A_CAST_: 0 = the activation codes and row scales are loaded as they are;
// 1 (FP32 scales) or 2 (power-of-two scales) = the activations arrive as BF16
// and are quantized on their way into LDS (ACaster).
// GATED_: the weights are F gate rows and F up rows ([2F][K], F a multiple of
// 128).  A wave's WN weight rows are WN/2 gate rows and the WN/2 up rows F
// further on; the tile's outputs are act(gate) * up, BN/2 columns.
constexpr int kOpFp8 = 0, kOpBf16 = 1, kOpWide16 = 2, kOpFp8Mx = 3;
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_, int ROWS_ = BM_,
          int PF_ = 0, int OP_ = kOpFp8, int W_ROWSCALE_ = 0, int A_CAST_ = 0, int GATED_ = 0>
struct GemmCfg {
  static constexpr bool GATED = GATED_ != 0;
  static constexpr bool OP_BF16 = OP_ == kOpBf16;
  static constexpr bool WIDE16 = OP_ == kOpWide16;
  static constexpr bool MX = OP_ == kOpFp8Mx;
  static constexpr bool W_ROWSCALE = W_ROWSCALE_ != 0;
  static constexpr bool A_CAST = A_CAST_ != 0;
  static constexpr int CAST_MODE = A_CAST ? A_CAST_ - 1 : 0;
  // MFMAs per 16x16 block per chunk
  static constexpr int SUB = OP_BF16 ? 2 : WIDE16 ? 4 : 1;
  static constexpr int BM = BM_;
  static constexpr int BN = BN_;
  static constexpr int BK = 128;                    // bytes of K per stage row and chunk
  static constexpr int WAVES_M = WAVES_M_;
  static constexpr int WAVES_N = WAVES_N_;
  static constexpr int NWAVES = WAVES_M * WAVES_N;
  static constexpr int THREADS = NWAVES * 64;
  static constexpr int WM = BM / WAVES_M;
  static constexpr int WN = BN / WAVES_N;
  static constexpr int MB = WM / 16;                // MFMA row blocks per wave
  static constexpr int NB = WN / 16;                // MFMA column blocks per wave
  static constexpr int ROWS = ROWS_;                // A rows staged per chunk (<= BM)
  static constexpr int A_BYTES = ROWS * BK;
  static constexpr int B_BYTES = BN * BK;
  static constexpr int SA_BYTES = OP_BF16 ? 0 : WAVES_M * 256;  // 64 row scales per row of waves
  // the tile's weight-row scales: 4 slots of 64 (rows past BN loaded, unused)
  static constexpr int SB_BYTES = W_ROWSCALE ? 4 * 256 : 0;
  static constexpr int STAGE = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
  static constexpr int STAGES = STAGES_;
  static constexpr int PF_LOADS = PF_;    // L2 prefetch loads per wave per chunk (0 or 1)
  static constexpr int PF_BYTES = PF_LOADS > 0 ? NWAVES * 256 : 0;  // their LDS landing slots
  static constexpr int LDS_BYTES = STAGE * STAGES + PF_BYTES;
  static constexpr int A_BLK = A_CAST ? 0 : A_BYTES / 1024;  // 1 KiB load instructions for A
  static constexpr int OP_BLK = A_BLK + B_BYTES / 1024;
  static constexpr int PER_WAVE = (OP_BLK + NWAVES - 1) / NWAVES;  // operand loads per wave
  static constexpr int PAD = PER_WAVE * NWAVES - OP_BLK;  // repeated A loads that even them out
  static constexpr int LOADS =
      PER_WAVE + (OP_BF16 || A_CAST ? 0 : 1) + (W_ROWSCALE ? 1 : 0);  // + scales
  static constexpr int CAST_ROUNDS = A_CAST ? (ROWS + 63) / 64 : 0;  // 64 rows per round
  static_assert(WM % 16 == 0 && WM <= 64, "a wave's rows fit one 256-byte scale slot");
  static_assert(W_ROWSCALE || 128 % WN == 0,
                "a wave's weight rows lie in one 128-row weight block (block-scaled weights)");
  // Staged rows: whole 1 KiB loads.  When they stop inside a wave (160 rows
  // in 48-row waves), that wave's fragment reads past them fall inside the
  // stage and feed only rows past the expert's end, which are not stored.
  static_assert(ROWS % 32 == 0 && ROWS <= BM, "staged rows fill whole loads within the tile");
  static_assert(PAD <= A_BLK, "the padding loads repeat A loads");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS budget");
  static_assert(STAGES >= 2 && STAGES <= 6, "ring depth");
  static_assert(PF_LOADS == 0 || (PF_LOADS == 1 && NWAVES >= 2 && ROWS == 256 && BN == 256),
                "the prefetch share is laid out for 256 x 256 tiles");
  static_assert(LOADS * (STAGES - 1) + PF_LOADS * (STAGES - 1) < 64, "vmcnt range");
  static_assert(!W_ROWSCALE || (!OP_BF16 && NWAVES == 8 && WAVES_N == 2 && BN <= 256),
                "row-scaled weights: 8 waves, each loading 64 of up to 256 row scales");
  static_assert(!A_CAST || (OP_ == kOpFp8 && !W_ROWSCALE && PF_LOADS == 0 && THREADS == 512 &&
                            A_CAST_ <= 2 && CAST_ROUNDS <= 4),
                "activation cast: 512 lanes, 8 per row, FP8 block-scaled weights");
  static_assert(OP_ >= kOpFp8 && OP_ <= kOpFp8Mx, "operand mode");
  static_assert(!MX || (!W_ROWSCALE && !A_CAST), "matrix-core scales: block-scaled dense GEMM");
  static_assert(!GATED || (OP_ == kOpFp8 && !W_ROWSCALE && !A_CAST && NB % 2 == 0 &&
                           (WN / 2) % 8 == 0 && 128 % (BN / 2) == 0),
                "gated block: FP8, block-scaled weights, one block of gate rows a tile");
};

// Main-loop schedule constants (measured on the 4096 x 4096 x 7168 shape;
// the result is insensitive to them within +-2%):
//   kDma0, kDmaStep  head load d of the next chunk goes out after MFMA
//                    kDma0 + d * kDmaStep;
//   kPromoteLag      a block's partial is promoted this many MFMAs after it
//                    was issued, when the matrix core has surely written it;
//   kBPrefetch       weight fragments are read this many row blocks ahead;
//   kBarLead         the chunk barrier sits this many MFMAs before the
//                    chunk's last row block.
//   kPfDist          the L2 prefetch issued while chunk g is computed
//                    touches chunk g + kPfDist.
constexpr int kPfDist = 6;
constexpr int kDma0 = 1;
constexpr int kDmaStep = 2;
constexpr int kPromoteLag = 2;
constexpr int kBPrefetch = 1;
constexpr int kBarLead = 2;

// Direct-to-LDS loads of one K chunk (A rows, W rows, row scales).  The
// operand tiles are cut into 1 KiB load instructions (8 rows of 128 B):
// instructions 0 .. A_BLK-1 carry A rows, the next ones W rows, and load d
// of wave w is instruction d*NWAVES + w, so every wave issues its share of
// the A rows first and then its share of the W rows (waves that issued only
// A or only W rows streamed the weights of the grouped tiles 1-2% slower);
// then comes the 256-byte slot of its row of waves' row scales (both waves
// of a row write the same values there): Cfg::LOADS instructions per wave
// per chunk.  When the operand loads do not split evenly over the waves, the
// last PAD instructions repeat the first A loads (same bytes to the same LDS
// place).  Lane
// i of an instruction lands at LDS byte 16*i, i.e. row i/8, physical column
// i%8, and so fetches logical column swz(row, i%8).  Rows past the valid range
// are clamped to the last valid row (their results are never stored).
//
// Addresses are buffer offsets: a scalar resource per operand based at the
// tile's first row, a per-lane 32-bit offset fixed for the whole tile, and the
// chunk's K offset as the scalar soffset, so issuing a load costs no VALU.
template <class Cfg>
struct ChunkLoader {
  __amdgpu_buffer_rsrc_t ra, rw, rs, rsb;
  __amdgpu_buffer_rsrc_t ru;  // gated: the up rows (rw: the gate rows)
  uint32_t voff[Cfg::PER_WAVE];
  uint32_t voff_s;
  uint32_t voff_sb;   // this lane's weight-row scale (row-scaled weights)
  int64_t sb_stride;  // bytes between consecutive chunks' weight-row scales
  uint32_t voff_pf;  // this lane's L2 prefetch line (first byte of its K chunk)
  bool pf_a;         // the wave prefetches A rows (else W rows)
  bool pf_up;        // gated: up rows of W
  int64_t s_stride;  // bytes between consecutive chunks' row scales
  int wave, wave_m;

  // Gated: whether row r of the tile's weight rows is an up row, and which of
  // the tile's gate (or up) rows it is.
  static __device__ __forceinline__ bool up_row(int r) { return r % Cfg::WN >= Cfg::WN / 2; }
  static __device__ __forceinline__ int half_row(int r) {
    return r / Cfg::WN * (Cfg::WN / 2) + r % (Cfg::WN / 2);
  }

  // Operand block of load instruction m (the padding repeats A blocks).
  static __device__ __forceinline__ int op_block(int m) {
    return m < Cfg::OP_BLK ? m : m - Cfg::OP_BLK;
  }

  __device__ __forceinline__ void init(const TileArgs& t, int wave_, int wave_m_, int lane) {
    wave = wave_;
    wave_m = wave_m_;
    const int64_t a_live = t.a_rows - t.a_row0;  // >= 1
    const int64_t w_live = t.w_rows - t.w_row0;  // >= 1
    if constexpr (!Cfg::A_CAST) ra = make_rsrc(t.A + t.a_row0 * t.K, a_live * t.K);
    rw = make_rsrc(t.W + t.w_row0 * t.K, w_live * t.K);
    if constexpr (Cfg::GATED) ru = make_rsrc(t.W + (t.w_rows + t.w_row0) * t.K, w_live * t.K);
    if constexpr (!Cfg::OP_BF16 && !Cfg::A_CAST) {
      const int64_t G = t.K / Cfg::BK;
      rs = make_rsrc(t.SA + t.a_row0, (G * t.sa_ld - t.a_row0) * 4);
      s_stride = t.sa_ld * 4;
    }
    const int sub_r = lane >> 3;
    const int pc = lane & 7;
#pragma unroll
    for (int j = 0; j < Cfg::PER_WAVE; ++j) {
      const int m = op_block(j * Cfg::NWAVES + wave);
      const bool is_a = m < Cfg::A_BLK;
      const int r = (is_a ? m : m - Cfg::A_BLK) * 8 + sub_r;
      const int64_t live = is_a ? a_live : w_live;
      const int src = Cfg::GATED && !is_a ? half_row(r) : r;  // row of the operand
      const int64_t rr = src < live ? src : live - 1;
      voff[j] = (uint32_t)(rr * t.K) + (uint32_t)(swz(r, pc) * 16);
    }
    // Lane i of the scale load fetches row (i & 3) * 16 + i / 4 of the wave's
    // rows (up to 64; rows past them are loaded and not used), so the scales
    // an MFMA column lane needs (rows c, 16 + c, 32 + c, 48 + c) sit side by
    // side in LDS.
    if constexpr (!Cfg::OP_BF16 && !Cfg::A_CAST) {
      const int64_t rs_row = wave_m_ * Cfg::WM + (lane & 3) * 16 + (lane >> 2);
      voff_s = (uint32_t)((rs_row < a_live ? rs_row : a_live - 1) * 4);
    }
    if constexpr (Cfg::W_ROWSCALE) {
      // Wave w loads the scales of weight rows 64*(w%4) .. +63 of the tile
      // (waves w and w+4 write the same values).
      const int64_t G = t.K / Cfg::BK;
      rsb = make_rsrc(t.SW + t.w_row0, (G * t.sw_ld - t.w_row0) * 4);
      sb_stride = t.sw_ld * 4;
      const int64_t sb_row = (wave_ % 4) * 64 + lane;
      voff_sb = (uint32_t)((sb_row < w_live ? sb_row : w_live - 1) * 4);
    }
    // L2 prefetch lines.  The XCD-aware tile order gives one XCD a block of
    // 4 tile rows x 8 tile columns, so 8 tiles share each 256-row A band and
    // 4 share each W band in that XCD's L2.  A tile therefore prefetches
    // only its share: A rows 32*(tn%8) .. +31 (wave 0, lanes 0..31) and W
    // rows 64*(tm%4) .. +63 (wave 1).  Every other lane repeats its wave's
    // first line, which the address unit merges into one request: a prefetch
    // costs 96 line requests per tile and chunk instead of 512.
    const int tm = (int)(t.a_row0 / Cfg::BM);
    const int tn = (int)(t.w_row0 / (Cfg::GATED ? Cfg::BN / 2 : Cfg::BN));
    pf_a = wave != 1;
    int pr = pf_a ? 32 * (tn % 8) : 64 * (tm % 4);
    // gated: the W share is 64 of the 128 gate rows or of the 128 up rows
    pf_up = Cfg::GATED && !pf_a && pr >= Cfg::BN / 2;
    if (pf_up) pr -= Cfg::BN / 2;
    if (wave == 1 || (wave == 0 && lane < 32)) pr += lane;
    const int64_t plive = pf_a ? a_live : w_live;
    voff_pf = (uint32_t)((pr < plive ? pr : plive - 1) * t.K);
  }

  // L2 prefetch h (0 .. PF_LOADS-1) of this lane's line of chunk g: a 4-byte
  // direct-to-LDS load into the wave's landing slot, whose contents nobody
  // reads.  It is counted by vmcnt like the operand loads.
  __device__ __forceinline__ void prefetch(uint8_t* slot, int64_t g, int h) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(pf_a ? ra : Cfg::GATED && pf_up ? ru : rw,
                                             to_lds(slot), 4,
                                             voff_pf + (uint32_t)(h * 64), (int)(g * Cfg::BK), 0, 0);
  }

  // Load d (0 .. LOADS-1) of chunk g into `stage`.
  __device__ __forceinline__ void issue(uint8_t* stage, int64_t g, int d) const {
    if (d < Cfg::PER_WAVE) {
      const int m = op_block(d * Cfg::NWAVES + wave);
      const bool is_a = m < Cfg::A_BLK;
      const int dst = is_a ? m * 1024 : Cfg::A_BYTES + (m - Cfg::A_BLK) * 1024;
      // (the 8 rows of an instruction are all gate or all up rows)
      const bool up = Cfg::GATED && !is_a && up_row((m - Cfg::A_BLK) * 8);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? ra : up ? ru : rw, to_lds(stage + dst), 16,
                                               voff[d], (int)(g * Cfg::BK), 0, 0);
    } else if (!Cfg::OP_BF16 && !Cfg::A_CAST && d == Cfg::PER_WAVE) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, to_lds(stage + Cfg::A_BYTES + Cfg::B_BYTES + wave_m * 256), 4, voff_s,
          (int)(g * s_stride), 0, 0);
    } else if constexpr (Cfg::W_ROWSCALE) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsb,
          to_lds(stage + Cfg::A_BYTES + Cfg::B_BYTES + Cfg::SA_BYTES + (wave % 4) * 256), 4,
          voff_sb, (int)(g * sb_stride), 0, 0);
    }
  }
};

// The activation operand quantized on its way into LDS: the FP8 cast fused
// with the global-to-LDS transfer (why-be.co.kr as_center post 57820,
// hardware-suggestion passage: the cast done during the transfer instead of
// an HBM round trip of the codes).  Each K chunk of the tile's BF16 rows
// comes into registers, 8 lanes per row (16 values, 32 bytes each) and 64
// rows per round (few registers: the main loop holds 221 of the 256).  The
// 8 lanes of a row reduce its 1x128 group max-abs (DPP), apply the
// quantizer's rule (quant_rules.hpp: the same codes and scale as
// fp8q_quantize_act, bit for bit), and write the codes into the stage's A
// slot at the swizzled places the direct loads would fill, and the scale into
// the row-scale slot of the row's wave row.  Rows past the valid range are
// read from the last valid row, as in the loads (their results are never
// stored).  The code has no branch: lanes past the staged
// rows (a partial last round) redo the last staged row and write the same
// bytes to the same places, and the 8 lanes of a row all write its scale.
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint16_t v2u16 __attribute__((ext_vector_type(2)));

// Max-abs of 16 BF16 values as BF16 magnitude bits (in the low half), by
// packed 16-bit integer max: for non-negative floats the integer order of the
// bit patterns is the numeric order, so this is exactly the max of |x|.
__device__ __forceinline__ uint32_t absmax16_bits(const uint4& p, const uint4& q) {
  const uint32_t m = 0x7FFF7FFFu;
  auto h = [](uint32_t w) { return __builtin_bit_cast(v2u16, w); };
  v2u16 r = __builtin_elementwise_max(h(p.x & m), h(p.y & m));
  r = __builtin_elementwise_max(r, __builtin_elementwise_max(h(p.z & m), h(p.w & m)));
  r = __builtin_elementwise_max(r, __builtin_elementwise_max(h(q.x & m), h(q.y & m)));
  r = __builtin_elementwise_max(r, __builtin_elementwise_max(h(q.z & m), h(q.w & m)));
  return r[0] > r[1] ? r[0] : r[1];
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
  return o > v ? o : v;
}

template <class Cfg>
struct ACaster {
  __amdgpu_buffer_rsrc_t rx;  // the tile's BF16 rows
  int a_last;                 // last valid row of the tile (only rows below ROWS matter)
  uint32_t row_bytes;         // 2K
  int row0;                   // this lane's row in round 0 (tid / 8)
  int oc;                     // which 16-value eighth of the row (= logical code column)
  uint4 raw[2];               // the loaded round's 16 BF16 values

  // LDS row of this lane in round r.
  __device__ __forceinline__ int row_of(int r) const {
    const int row = r * 64 + row0;
    return row < Cfg::ROWS ? row : Cfg::ROWS - 1;
  }

  __device__ __forceinline__ void init(const TileArgs& t, int tid) {
    const int64_t a_live = t.a_rows - t.a_row0;  // >= 1
    rx = make_rsrc(t.A + t.a_row0 * 2 * t.K, a_live * 2 * t.K);
    a_last = (int)(a_live < Cfg::ROWS ? a_live - 1 : Cfg::ROWS - 1);
    row_bytes = (uint32_t)(2 * t.K);
    row0 = tid >> 3;
    oc = tid & 7;
  }

  // BF16 values of chunk g, round r, into registers.
  __device__ __forceinline__ void load(int64_t g, int r) {
    const int row = row_of(r);
    const uint32_t rr = (uint32_t)(row < a_last ? row : a_last);
    const uint32_t voff = rr * row_bytes + (uint32_t)(oc * 32);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const v4u v = __builtin_amdgcn_raw_buffer_load_b128(rx, voff + (uint32_t)(16 * p),
                                                         (int)(g * 256), 0);
      raw[p] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }

  // Codes and scale of the loaded round r into `stage`.
  __device__ __forceinline__ void cast_store(uint8_t* stage, int r) const {
    uint32_t ab = absmax16_bits(raw[0], raw[1]);
    ab = dpp_umax<kDppQuadXor1>(ab);       // the 8 lanes of a row: two quads,
    ab = dpp_umax<kDppQuadXor2>(ab);
    ab = dpp_umax<kDppRowHalfMirror>(ab);  // then each quad against the other
    const GroupRule rule = group_rule<Cfg::CAST_MODE>(__uint_as_float(ab << 16));
    const uint2 c0 = convert8<Cfg::CAST_MODE>(raw[0], rule);
    const uint2 c1 = convert8<Cfg::CAST_MODE>(raw[1], rule);
    const int row = row_of(r);
    // K bytes 16oc .. 16oc+15 of the row: logical 16-byte column oc.
    *reinterpret_cast<v4u*>(stage + row * 128 + swz(row, oc) * 16) = v4u{c0.x, c0.y, c1.x, c1.y};
    // Slot position of row rr of a wave row: (rr % 16) * 4 + rr / 16, the
    // order the scale loads of the other configurations produce.
    const int wm = row / Cfg::WM, rr = row % Cfg::WM;
    *reinterpret_cast<float*>(stage + Cfg::A_BYTES + Cfg::B_BYTES + wm * 256 +
                              ((rr & 15) * 4 + (rr >> 4)) * 4) = rule.s;
  }
};

// One 32-K half of a chunk for BF16 operands: fragment half h (the 16-byte
// piece q, or q + 4, of the 128-byte row, i.e. 8 BF16 values per lane) of the
// weight and activation fragments, accumulated into acc by the matrix core.
__device__ __forceinline__ v4f mfma_bf16_half(const v8i& w, const v8i& a, const v4f& acc,
                                              int h) {
  typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
  const v4i wh = h ? v4i{w[4], w[5], w[6], w[7]} : v4i{w[0], w[1], w[2], w[3]};
  const v4i ah = h ? v4i{a[4], a[5], a[6], a[7]} : v4i{a[0], a[1], a[2], a[3]};
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, wh),
                                                 __builtin_bit_cast(v8bf, ah), acc, 0, 0, 0);
}

// Promotion with row-scaled weights: acc += P * (s_a[row] * s_b[col]), the
// lane's 4 results having 4 weight rows.
__device__ __forceinline__ void promote_rows(v4f& acc, const v4f& p, float sa, const v4f& sb) {
  acc[0] = __builtin_fmaf(p[0], sa * sb[0], acc[0]);
  acc[1] = __builtin_fmaf(p[1], sa * sb[1], acc[1]);
  acc[2] = __builtin_fmaf(p[2], sa * sb[2], acc[2]);
  acc[3] = __builtin_fmaf(p[3], sa * sb[3], acc[3]);
}

// Promotion of one 16x16 chunk partial: acc += P * (s_a[row] * s_w).
__device__ __forceinline__ void promote(v4f& acc, const v4f& p, float mult) {
  acc[0] = __builtin_fmaf(p[0], mult, acc[0]);
  acc[1] = __builtin_fmaf(p[1], mult, acc[1]);
  acc[2] = __builtin_fmaf(p[2], mult, acc[2]);
  acc[3] = __builtin_fmaf(p[3], mult, acc[3]);
}

// Precise mode.  A fragment's 32 E4M3 codes widened to FP16, exactly (every
// E4M3 value, subnormals included, is an FP16 value; the conversion's scale
// operand 1.0 leaves it unscaled): FP16 word 2d + s holds byte 2s, 2s + 1 of
// code word d.  Quarter h (FP16 words 4h .. 4h+3) is fragment bytes 8h .. 8h+7,
// the 8 K values one lane gives one 16x16x32 MFMA; weight and activation
// quarters pair the same K.
typedef int v16i __attribute__((ext_vector_type(16)));
__device__ __forceinline__ v4i widen_quarter(const v8i& f, int h) {
  v4i o;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const int w = f[2 * h + d];
    o[2 * d] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
    o[2 * d + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
  }
  return o;
}

__device__ __forceinline__ v16i widen_frag(const v8i& f) {
  v16i o;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const v4i x = widen_quarter(f, h);
    o[4 * h] = x[0];
    o[4 * h + 1] = x[1];
    o[4 * h + 2] = x[2];
    o[4 * h + 3] = x[3];
  }
  return o;
}

__device__ __forceinline__ v4i quarter(const v16i& f, int h) {
  return v4i{f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]};
}

// One 32-K quarter of a chunk on widened codes: c + W_quarter . A_quarter.
__device__ __forceinline__ v4f mfma_wide16(const v4i& w, const v4i& a, const v4f& c) {
  typedef _Float16 v8h __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, w),
                                                __builtin_bit_cast(v8h, a), c, 0, 0, 0);
}


// Block-scaled FP8 MFMA from zero: weight operand scaled by 2^(sw - 127),
// activation operand by 2^(byte i of sa - 127) (E8M0 bytes; op_sel picks the
// byte, so it must be an immediate: i is 0..3).
__device__ __forceinline__ v4f mfma_mx(const v8i& w, const v8i& a, int sw, int sa, int i) {
  const v4f z = {0.f, 0.f, 0.f, 0.f};
  switch (i) {
    case 0: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, z, 0, 0, 0, sw, 0, sa);
    case 1: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, z, 0, 0, 0, sw, 1, sa);
    case 2: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, z, 0, 0, 0, sw, 2, sa);
    default: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, z, 0, 0, 0, sw, 3, sa);
  }
}

// E8M0 byte of a power-of-two scale s >= 0 and the factor the matrix core
// cannot take: a normal s = 2^e is byte e + 127 (its FP32 exponent field) with
// factor 1; a subnormal s (e < -126) takes byte 0 (2^-127) and the exact
// factor s * 2^127; s = 0 (a flushed group, all codes zero) gives factor 0.
__device__ __forceinline__ int e8m0_byte(float s, float& factor) {
  const int b = (__float_as_int(s) >> 23) & 0xFF;
  factor = b == 0 ? s * 0x1p127f : 1.0f;
  return b;
}

// Computes one BM x BN output tile.  All lanes of the workgroup call it.
template <class Cfg>
__device__ __forceinline__ void gemm_tile(const TileArgs& t, uint8_t* smem) {
  constexpr int MB = Cfg::MB, NB = Cfg::NB, S = Cfg::STAGES;
  constexpr int RB = MB * Cfg::SUB;  // MFMA steps per weight row block
  constexpr bool WIDE = Cfg::WIDE16;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave_m = wave / Cfg::WAVES_N;
  const int wave_n = wave % Cfg::WAVES_N;
  const int r16 = lane & 15;   // fragment row within a 16-row block
  const int q = lane >> 4;     // which 16-byte piece pair of the 128-byte chunk
  const int64_t G = t.K / Cfg::BK;

  // Weight-scale row of this wave's weight rows (one 128-row block).
  const float* sw_row = nullptr;
  const float* sw_up = nullptr;  // gated: of its up rows (sw_row: of its gate rows)
  if constexpr (Cfg::GATED) {
    sw_row = t.SW + (t.w_row0 + wave_n * (Cfg::WN / 2)) / 128 * G;
    sw_up = sw_row + t.w_rows / 128 * G;
  } else if constexpr (!Cfg::OP_BF16 && !Cfg::W_ROWSCALE) {
    int64_t wblk = (t.w_row0 + wave_n * Cfg::WN) / 128;
    const int64_t last_wblk = t.w_rows / 128 - 1;
    wblk = wblk < last_wblk ? wblk : last_wblk;
    sw_row = t.SW + wblk * G;
  }

  // Waves whose rows are all past the valid range skip the MFMA work.
  const bool wave_live =
      (wave_m * Cfg::WM < Cfg::ROWS) && (t.a_row0 + wave_m * Cfg::WM) < t.a_rows;

  // acc[i][j]: activation row block i (16 rows) x weight row block j.
  v4f acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // Schedule of one chunk g (k = MFMA index, LAG = promotion lag):
  //   k = 0 ..         MFMAs of chunk g; the head loads of chunk g+S-1 go out
  //                    one every kDmaStep MFMAs from k = kDma0;
  //   k = kBar         wait for chunk g+1's loads, barrier: every wave has
  //                    finished reading stage g (its last weight fragment was
  //                    read at k = MB*(NB-1-BPF)) and chunk g+1 is in LDS;
  //   k > kBar         the tail loads of chunk g+S go into stage g, one per
  //                    MFMA, and once a fragment register has served its last
  //                    MFMA of chunk g it is refilled with chunk g+1's data,
  //                    so chunk g+1 starts with its operands in registers.
  // Step k is MFMA (weight row block j = k / MB, activation block i = k % MB):
  // one weight fragment serves MB consecutive MFMAs.  With BF16 operands a
  // block takes SUB = 2 MFMAs per chunk (the chunk's two 32-K halves): row
  // block j runs steps RB*j .. RB*j + RB - 1, first half h = 0 for the MB
  // activation blocks, then h = 1, so chained MFMAs are MB steps apart.
  // The matrix core therefore never waits for a chunk boundary: a wave that
  // arrives early at the barrier leaves the matrix core to its SIMD partner.
  // (Lag 1 with the activation cast: its registers come out of the partials'.)
  // In the precise mode (WIDE) a block's SUB = 4 MFMAs are consecutive steps
  // chained through their C operand (block b = k / SUB, i.e. activation block
  // i = b % MB of weight row block j = b / MB, quarter h = k % SUB); the
  // weight fragment of row block j is widened quarter by quarter in the steps
  // of its first block, and block b is promoted LAG steps after its last MFMA.
  constexpr int LAG = Cfg::OP_BF16 ? 0 : Cfg::A_CAST ? 1 : kPromoteLag;
  static_assert(!WIDE || LAG < Cfg::SUB, "two partial registers serve the precise mode");
  constexpr int KSTEPS = RB * NB + LAG;
  constexpr int kBar = RB * (NB - 1) - kBarLead;   // before the last row block
  constexpr int TAIL = KSTEPS - 1 - kBar;          // loads issued after the barrier
  constexpr int D1 = TAIL < Cfg::LOADS ? TAIL : Cfg::LOADS;
  // Weight fragments are read BPF row blocks ahead into a ring of BPF+1 slots.
  constexpr int BPF = kBPrefetch;
  constexpr int NBUF = BPF + 1;
  static_assert(kBar > RB * (NB - 1 - BPF), "the barrier follows the last weight read");
  static_assert(kBar < RB * (NB - 1), "the barrier precedes the last row block");
  // Step after which weight slot t (t < BPF) is free for chunk g+1's block t: the
  // last MFMA of the last block j < NB with j % NBUF == t, but not before the
  // barrier.
  auto next_b_step = [](int t) constexpr {
    int jt = t;
    while (jt + NBUF < NB) jt += NBUF;
    const int kt = RB * jt + RB - 1;
    return kt > kBar ? kt : kBar;
  };
  static_assert(kDma0 + (Cfg::LOADS - D1 - 1) * kDmaStep < kBar,
                "head loads are issued before the barrier");
  // The prefetches follow the head loads, kDmaStep MFMAs apart.
  constexpr int kPfAt = kDma0 + (Cfg::LOADS - D1) * kDmaStep;
  static_assert(kPfAt > kDma0 + (Cfg::LOADS - D1 - 1) * kDmaStep &&
                    kPfAt + (Cfg::PF_LOADS - 1) * kDmaStep < kBar,
                "prefetches go out after the head loads and before the barrier");

  // Activation cast: round r of chunk g+1 is quantized into chunk g+1's stage
  // at step cast_step(r) of chunk g, the last one a few steps before the
  // barrier that publishes chunk g+1.  Round 0's BF16 values are loaded right after
  // chunk g-1's barrier, ahead of the operand loads issued there, and round
  // r+1's right after round r's cast (one register set: a second one spills
  // the main loop), so each load has the steps up to its cast to arrive; the
  // casts are spread evenly over the chunk's cycle.  The stage of chunk g+1 is
  // free from chunk g's start on: its last reader, chunk g+1-S, ended before
  // chunk g-1's barrier.
  constexpr int CR = Cfg::CAST_ROUNDS;
  constexpr int kCastLast = kBar - 3;
  constexpr int kCastGap =
      CR > 1 ? (kCastLast / (CR - 1) < KSTEPS / CR ? kCastLast / (CR - 1) : KSTEPS / CR) : 0;
  auto cast_step = [](int r) constexpr { return kCastLast - (CR - 1 - r) * kCastGap; };
  static_assert(CR == 0 || (cast_step(0) >= 0 && kBar + 1 < KSTEPS),
                "the casts of a chunk precede its barrier");

  ChunkLoader<Cfg> ld;
  ld.init(t, wave, wave_m, lane);
  ACaster<Cfg> cs;
  if constexpr (Cfg::A_CAST) cs.init(t, threadIdx.x);
  // Chunk indices past the end are clamped to the last chunk: the extra loads
  // re-fetch L2-resident bytes into a stage nobody reads again, and keep the
  // number of loads in flight the same every iteration.
  const int64_t g_last = G - 1;
  uint8_t* const pf_slot = smem + S * Cfg::STAGE + wave * 256;
  constexpr int PFL = Cfg::PF_LOADS;
  // Loads issued after the last load of the chunk a barrier waits for: in
  // steady state S-2 whole chunks and S-1 iterations' prefetches.
  constexpr int kAfter = Cfg::LOADS * (S - 2) + PFL * (S - 1);
  // The prologue issues chunks 0 .. S-2 and the first D1 loads of chunk S-1
  // in the order S-1 steady-state iterations would (each chunk followed by
  // one iteration's prefetches), so every wait below counts the same loads.
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
#pragma unroll
    for (int d = 0; d < Cfg::LOADS; ++d)
      ld.issue(smem + s * Cfg::STAGE, s < g_last ? s : g_last, d);
    const int64_t gp = s - (S - 1) + kPfDist;
#pragma unroll
    for (int h = 0; h < PFL; ++h)
      ld.prefetch(pf_slot, gp < 0 ? 0 : (gp < g_last ? gp : g_last), h);
  }
#pragma unroll
  for (int d = 0; d < D1; ++d)
    ld.issue(smem + (S - 1) * Cfg::STAGE, S - 1 < g_last ? S - 1 : g_last, d);
  if constexpr (Cfg::A_CAST) {
#pragma unroll
    for (int r = 0; r < CR; ++r) {
      cs.load(0, r);
      cs.cast_store(smem, r);
    }
  }
  wait_vmcnt<kAfter + D1>();  // chunk 0 landed
  lds_barrier();
  if constexpr (Cfg::A_CAST) cs.load(g_last > 0 ? 1 : 0, 0);

  // activation fragments of the chunk (MFMA B operand); widened to FP16 in
  // the precise mode
  using AFrag = typename std::conditional<WIDE, v16i, v8i>::type;
  AFrag a[MB];
  v8i b[NBUF];   // weight fragments, a ring over row blocks (MFMA A operand)
  v16i bw;       // precise mode: the current row block's weight fragment, widened
  if (wave_live) {
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      if constexpr (WIDE)
        a[i] = widen_frag(load_frag(smem, wave_m * Cfg::WM + i * 16 + r16, q));
      else
        a[i] = load_frag(smem, wave_m * Cfg::WM + i * 16 + r16, q);
    }
#pragma unroll
    for (int t = 0; t < BPF; ++t)
      b[t] = load_frag(smem + Cfg::A_BYTES, wave_n * Cfg::WN + t * 16 + r16, q);
  }

  int cur = 0;  // stage of chunk g
  for (int64_t g = 0; g < G; ++g) {
    const int nxt = cur + 1 == S ? 0 : cur + 1;    // stage of chunk g+1
    const int head = cur == 0 ? S - 1 : cur - 1;   // stage of chunk g+S-1
    const int64_t g_head = g + S - 1 < g_last ? g + S - 1 : g_last;
    const int64_t g_tail = g + S < g_last ? g + S : g_last;
    const int64_t g_pf = g + kPfDist < g_last ? g + kPfDist : g_last;
    const int64_t g_nxt = g + 1 < g_last ? g + 1 : g_last;
    const int64_t g_nxt2 = g + 2 < g_last ? g + 2 : g_last;
    uint8_t* const st_cur = smem + cur * Cfg::STAGE;
    uint8_t* const st_nxt = smem + nxt * Cfg::STAGE;
    uint8_t* const st_head = smem + head * Cfg::STAGE;
    if (!wave_live) {
#pragma unroll
      for (int d = D1; d < Cfg::LOADS; ++d) ld.issue(st_head, g_head, d);
#pragma unroll
      for (int h = 0; h < PFL; ++h) ld.prefetch(pf_slot, g_pf, h);
      if constexpr (Cfg::A_CAST) {
#pragma unroll
        for (int r = 0; r < CR; ++r) {
          cs.cast_store(st_nxt, r);
          if (r + 1 < CR) cs.load(g_nxt, r + 1);
        }
      }
      wait_vmcnt<kAfter>();
      lds_barrier();
      if constexpr (Cfg::A_CAST) cs.load(g_nxt2, 0);
#pragma unroll
      for (int d = 0; d < D1; ++d) ld.issue(st_cur, g_tail, d);
      cur = nxt;
      continue;
    }

    const uint8_t* Bs = st_cur + Cfg::A_BYTES;
    float mult[MB];
    float mult_up[MB];  // gated: the up rows' multipliers
    int mx_w = 0, mx_a = 0;  // matrix-core scales: E8M0 bytes (weights; 4 activation blocks)
    v4f sa;
    // Row-scaled weights: the scales of row block j (this lane's 4 weight
    // rows) go into a 3-slot ring when the block's fragment is prefetched;
    // its last promotion comes before the slot is reused.
    const float* SBs =
        reinterpret_cast<const float*>(st_cur + Cfg::A_BYTES + Cfg::B_BYTES + Cfg::SA_BYTES);
    v4f sbv[3];
    if constexpr (!Cfg::OP_BF16) {
      const float* SAs =
          reinterpret_cast<const float*>(st_cur + Cfg::A_BYTES + Cfg::B_BYTES + wave_m * 256);
      sa = *reinterpret_cast<const v4f*>(SAs + 4 * r16);
      if constexpr (Cfg::W_ROWSCALE) {
        sbv[0] = *reinterpret_cast<const v4f*>(SBs + wave_n * Cfg::WN + 4 * q);
      } else if constexpr (Cfg::MX) {
        static_assert(MB <= 4, "one byte per activation block in a 32-bit scale register");
        float fw;
        mx_w = e8m0_byte(sw_row[g], fw);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          float fa;
          mx_a |= e8m0_byte(sa[i], fa) << (8 * i);
          mult[i] = fa * fw;   // 1 unless a scale is below 2^-126
        }
      } else {
        const float sw = sw_row[g];
#pragma unroll
        for (int i = 0; i < MB; ++i) mult[i] = sa[i] * sw;
        if constexpr (Cfg::GATED) {
          const float su = sw_up[g];
#pragma unroll
          for (int i = 0; i < MB; ++i) mult_up[i] = sa[i] * su;
        }
      }
    }
    // chunk partials: a ring over steps, or over blocks in the precise mode
    constexpr int PN = WIDE ? 2 : LAG + 1;
    v4f p[PN];
#pragma unroll
    for (int k = 0; k < KSTEPS; ++k) {
      if (k < RB * NB) {
        const int i = WIDE ? (k / Cfg::SUB) % MB : k % MB;
        const int h = WIDE ? k % Cfg::SUB : (k / MB) % Cfg::SUB;
        const int j = k / RB;
        if (k % RB == 0 && j + BPF < NB)
          b[(j + BPF) % NBUF] = load_frag(Bs, wave_n * Cfg::WN + (j + BPF) * 16 + r16, q);
        if constexpr (Cfg::W_ROWSCALE) {
          static_assert(RB * (NB - 2) < kBar, "row scales are read before the barrier");
          if (k % RB == 0 && j + 1 < NB)
            sbv[(j + 1) % 3] =
                *reinterpret_cast<const v4f*>(SBs + wave_n * Cfg::WN + (j + 1) * 16 + 4 * q);
        }
        if constexpr (Cfg::OP_BF16) {
          acc[i][j] = mfma_bf16_half(b[j % NBUF], a[i], acc[i][j], h);
        } else if constexpr (WIDE) {
          if (i == 0) {
            const v4i x = widen_quarter(b[j % NBUF], h);
            bw[4 * h] = x[0];
            bw[4 * h + 1] = x[1];
            bw[4 * h + 2] = x[2];
            bw[4 * h + 3] = x[3];
          }
          const int pb = (k / Cfg::SUB) % 2;
          p[pb] = mfma_wide16(quarter(bw, h), quarter(a[i], h),
                              h == 0 ? v4f{0.f, 0.f, 0.f, 0.f} : p[pb]);
        } else if constexpr (Cfg::MX) {
          p[k % (LAG + 1)] = mfma_mx(b[j % NBUF], a[i], mx_w, mx_a, i);
        } else {
          p[k % (LAG + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              b[j % NBUF], a[i], v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int d = D1; d < Cfg::LOADS; ++d)
        if (k == kDma0 + (d - D1) * kDmaStep) ld.issue(st_head, g_head, d);
#pragma unroll
      for (int h = 0; h < PFL; ++h)
        if (k == kPfAt + h * kDmaStep) ld.prefetch(pf_slot, g_pf, h);
      if (k == kBar) {
        wait_vmcnt<kAfter>();  // chunk g+1 landed
        lds_barrier();
      }
      if (k < RB * NB) {
        // Chunk g+1's fragments go into registers as soon as their chunk-g
        // contents have served their last MFMA (and the barrier at kBar has
        // made chunk g+1 visible): a[i] after row block NB-1's last MFMA with
        // it, weight slot t after the last block of chunk g that uses it.
        const int i = WIDE ? (k / Cfg::SUB) % MB : k % MB;
        const int h = WIDE ? k % Cfg::SUB : (k / MB) % Cfg::SUB;
        const int j = k / RB;
        if (j == NB - 1 && h == Cfg::SUB - 1) {
          if constexpr (WIDE)
            a[i] = widen_frag(load_frag(st_nxt, wave_m * Cfg::WM + i * 16 + r16, q));
          else
            a[i] = load_frag(st_nxt, wave_m * Cfg::WM + i * 16 + r16, q);
        }
#pragma unroll
        for (int t = 0; t < BPF; ++t)
          if (k == next_b_step(t))
            b[t] = load_frag(st_nxt + Cfg::A_BYTES, wave_n * Cfg::WN + t * 16 + r16, q);
      }
      // (Issued before the tail loads, so that waiting for these BF16
      // values never waits for chunk g+S's operands.)
      if constexpr (Cfg::A_CAST)
        if (k == kBar + 1) cs.load(g_nxt2, 0);
#pragma unroll
      for (int d = 0; d < D1; ++d)
        if (k == kBar + 1 + d) ld.issue(st_cur, g_tail, d);
      // Keep the step order: MFMA k is issued before block k-LAG's
      // promotion.  Left free, the scheduler hoists the promotion above the
      // MFMA (to hand its result registers to MFMA k), which leaves it right
      // behind MFMA k-LAG+1 and stalls the wave on the matrix core's result.
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (WIDE) {
        // block bb's last MFMA was step kp
        const int kp = k - LAG;
        if (kp >= 0 && kp < RB * NB && kp % Cfg::SUB == Cfg::SUB - 1) {
          const int bb = kp / Cfg::SUB;
          if constexpr (Cfg::W_ROWSCALE)
            promote_rows(acc[bb % MB][bb / MB], p[bb % 2], sa[bb % MB], sbv[(bb / MB) % 3]);
          else
            promote(acc[bb % MB][bb / MB], p[bb % 2], mult[bb % MB]);
        }
      } else if constexpr (Cfg::W_ROWSCALE) {
        const int kp = k - LAG;
        if (kp >= 0)
          promote_rows(acc[kp % MB][kp / MB], p[kp % (LAG + 1)], sa[kp % MB], sbv[(kp / MB) % 3]);
      } else if constexpr (!Cfg::OP_BF16) {
        const int kp = k - LAG;
        if (kp >= 0)
          promote(acc[kp % MB][kp / MB], p[kp % (LAG + 1)],
                  Cfg::GATED && kp / MB >= NB / 2 ? mult_up[kp % MB] : mult[kp % MB]);
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (Cfg::A_CAST) {
#pragma unroll
        for (int r = 0; r < CR; ++r)
          if (k == cast_step(r)) {
            cs.cast_store(st_nxt, r);
            if (r + 1 < CR) cs.load(g_nxt, r + 1);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    cur = nxt;
  }
  wait_vmcnt<0>();  // the trailing (clamped) loads have landed before the waves exit

  // Epilogue: in block (i, j) the lane holds activation row m = 16i + r16 and
  // weight rows n = 16j + 4q .. 16j + 4q + 3, i.e. 4 consecutive outputs.
  if constexpr (Cfg::GATED) {
    // Blocks j < NB/2 are gate rows, block j + NB/2 the matching up rows.  The
    // outputs of 16 activation rows pass through the wave's share of the ring,
    // from which 16-byte pieces of whole row runs are stored (4096 tokens, F =
    // 2048, K = 7168: 101 us, 108 with Y saved; the lanes' own 8-byte pieces
    // stored as they are 104 and 118).
    lds_barrier();  // the ring is free
    if (!wave_live) return;
    constexpr int NO = NB / 2;
    uint8_t* const mine = smem + wave * (Cfg::LDS_BYTES / Cfg::NWAVES / 16 * 16);
    static_assert(Cfg::LDS_BYTES / Cfg::NWAVES >= 16 * (64 * NO + 16) + 16, "16 rows of FP32 fit");
    const int64_t col = t.w_row0 + wave_n * (Cfg::WN / 2);
    auto put = [&](const v4f(&v)[NO], auto bf16, void* out, int64_t row0, int64_t ld, int64_t c0) {
      constexpr int OB = decltype(bf16)::value ? 2 : 4, ROW = 16 * NO * OB, PITCH = ROW + 16;
#pragma unroll
      for (int j = 0; j < NO; ++j) {
        uint8_t* const at = mine + r16 * PITCH + (16 * j + 4 * q) * OB;
        if constexpr (OB == 2)
          *reinterpret_cast<uint2*>(at) =
              make_uint2(pack_bf16x2(v[j][0], v[j][1]), pack_bf16x2(v[j][2], v[j][3]));
        else
          *reinterpret_cast<v4f*>(at) = v[j];
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int x0 = 0; x0 < ROW; x0 += 64) {  // 16 rows of ROW/16 pieces
        const int r = (x0 + lane) / (ROW / 16), c = (x0 + lane) % (ROW / 16);
        if (r < 16 && row0 + r < t.a_rows)
          *reinterpret_cast<v4u*>(static_cast<uint8_t*>(out) + ((row0 + r) * ld + c0) * OB +
                                  16 * c) = *reinterpret_cast<const v4u*>(mine + r * PITCH + 16 * c);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int64_t row0 = t.a_row0 + wave_m * Cfg::WM + 16 * i;
      v4f g[NO], u[NO], h[NO];
#pragma unroll
      for (int j = 0; j < NO; ++j) {
        g[j] = acc[i][j];
        u[j] = acc[i][j + NO];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[j][e] = act_fast(t.act, g[j][e]) * u[j][e];
      }
      if (t.out_bf16)
        put(h, std::true_type{}, t.C, row0, t.ldc, col);
      else
        put(h, std::false_type{}, t.C, row0, t.ldc, col);
      if (t.gu) {
        put(g, std::true_type{}, t.gu, row0, 2 * t.ldc, col);
        put(u, std::true_type{}, t.gu, row0, 2 * t.ldc, t.ldc + col);
      }
    }
    return;
  }
  if (!wave_live) return;
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int64_t m = t.a_row0 + wave_m * Cfg::WM + i * 16 + r16;
    if (m >= t.a_rows) continue;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t n = t.w_row0 + wave_n * Cfg::WN + j * 16 + 4 * q;
      if (n >= t.w_rows) continue;
      if (t.out_bf16) {
        uint2 o;
        o.x = f32_to_bf16_bits(acc[i][j][0]) | (f32_to_bf16_bits(acc[i][j][1]) << 16);
        o.y = f32_to_bf16_bits(acc[i][j][2]) | (f32_to_bf16_bits(acc[i][j][3]) << 16);
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(t.C) + m * t.ldc + n) = o;
      } else {
        *reinterpret_cast<v4f*>(reinterpret_cast<float*>(t.C) + m * t.ldc + n) = acc[i][j];
      }
    }
  }
}

}  // namespace fp8q
