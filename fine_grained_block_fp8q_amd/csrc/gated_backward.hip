// Backward pass of the gated activation, quantized for the two gradient GEMMs.
//
// For h = act(gate) * up with Y = [gate | up] = X W^T:
//   dgate = dh * up * act'(gate),   dup = dh * act(gate),   dY = [dgate | dup];
//   dX = dY W     takes dY in 1x128 groups along the 2F features (q, s),
//   dW = dY^T X   takes dY^T in groups of 128 tokens             (qt, st).
// Both forms come from one pass: dh, gate and up are read once (6 bytes a
// feature), dY stays in FP32 registers and is never rounded to BF16, and each
// form of its codes is written once (2 + 2 bytes): bound by memory.
//
// A workgroup of 512 lanes takes 128 tokens x 128 features, so that it holds
// whole groups in both directions.  Lane (rq = t/16, l16 = t%16) owns tokens
// 4rq .. 4rq+3 at features 8 l16 .. 8 l16 + 7.  A row group's maximum is one
// DPP row's; a column group's goes over the lane's 4 tokens, the wave's 4 rq
// (shuffles) and the 8 waves (LDS).  Each group's rule (two divisions) is
// worked out by one lane, not by all that hold the group: lane i of a DPP row
// takes row group i of its 8 and broadcasts the multiplier.  The lane's 4
// tokens of one feature are one word of the transposed codes, which are
// gathered in LDS and stored 128 bytes (a feature's group of tokens) to 8 lanes.
//
// 4000 tokens, F = 2048: 16.2 us for 82 MB (5.1 TB/s, a large copy's rate); the
// rows' form alone 12.4, the tokens' alone 14.1.  With the library's exponential,
// correctly rounded divisions by every lane and branches for the last tokens it
// was 22.2, bound by the vector ALU.
//
// A single such workgroup takes 5 us of its 1580 vector instructions, while most
// CUs have none.  With few groups each form is therefore formed by itself, in
// pieces of 16 tokens or of 32 features (a quarter and an eighth of the work of
// a block), and the operands are read twice.  Both forms, us, blocks of 128 x 128:
//   blocks         16    32    64    128   256   512
//   one pass       8.8   8.9   9.1   9.3   10.1  16.7
//   small pieces   4.4   4.9   5.8   8.4   18.4  31.6
// of which 3.5 is a launch.  Up to 128 blocks the small pieces are taken.
//
// Tokens past M count as zeros: the last group of tokens is a full one, and its
// codes past M are zero.
//
// By expert (EXPERTS): the groups of tokens are those of experts.hpp, of which each
// expert's last one may end early; everything else is the same.  Rows past the
// last expert are in no group, and their codes along the features not written.
// Finding a group's rows takes as long as a fifth of a block, so a workgroup takes
// several blocks of features; waves without tokens and groups that there are not are
// spared the work.  F = 2048, us, before and after: 8192 tokens of 32 experts 45.6 and
// 41, 32768 of 256 (groups two thirds full) 260 and 205, 2000 of 64 32 and 20.6.

#include <type_traits>

#include "activation.hpp"
#include "experts.hpp"
#include "gemm_common.hpp"
#include "launch.hpp"
#include "quant_rules.hpp"

namespace fp8q {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kBwThreads = 512;

// Few groups: up to so many 128 x 128 blocks each form has workgroups of its
// own, of 16 tokens (rows' form) and 32 features (tokens' form).
constexpr int kRowsTokens = 16, kTokensFeatures = 32, kSmallThreads = 256;
constexpr int64_t kSmallBlocks = 128;
// By expert a workgroup takes up to kBwBlocks blocks of features, as many as leave
// kBwWorkgroups of them.
constexpr int64_t kBwBlocks = 4, kBwWorkgroups = 2048;

__device__ __forceinline__ float bf16_elem(const uint4& v, int j) {
  const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
  return (j & 1) ? bf16_hi(w) : bf16_lo(w);
}

constexpr int kNonTemporal = 2;  // cache policy bit of a buffer store

__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  const v4u v = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
  return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ uint4 load8(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  const v2u v = __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
  return make_uint4(v[0], v[1], 0, 0);
}

// dgate and dup of element j of dh, gate and up.
template <int ACT>
__device__ __forceinline__ void gate_up_grad(const uint4& dh, const uint4& gate, const uint4& up,
                                             int j, float& dg, float& du) {
  const float x = bf16_elem(dh, j);
  float a, da;
  act_and_grad(ACT, bf16_elem(gate, j), a, da);
  dg = x * bf16_elem(up, j) * da;
  du = x * a;
}

// LDS byte of token word rq (tokens 4rq..4rq+3) of feature c in a transposed
// tile: rows of 128 bytes whose 16-byte pieces are exchanged by the feature's
// octet, so that the 16 l16 of a wave write 8 different pieces.
__device__ __forceinline__ int tile_at(int c, int rq) {
  return c * 128 + (((rq >> 2) ^ (c >> 3)) & 7) * 16 + (rq & 3) * 4;
}

// What apply() needs of a rule, in 32 bits: the multiplier or the exponent.
template <int MODE>
__device__ __forceinline__ float rule_word(const GroupRule& r) {
  return MODE == 0 ? r.mul : __int_as_float(r.neg_e);
}
template <int MODE>
__device__ __forceinline__ GroupRule word_rule(float w) {
  GroupRule r;
  r.mul = MODE == 0 ? w : 0.f;
  r.neg_e = MODE == 0 ? 0 : __float_as_int(w);
  r.s = 0.f;
  return r;
}

// The rule that lane N of this DPP row (16 lanes) holds.
template <int MODE, int N>
__device__ __forceinline__ GroupRule rule_of_lane(const GroupRule& r) {
  constexpr int kRowNewBcast = 0x150;
  return word_rule<MODE>(__int_as_float(__builtin_amdgcn_update_dpp(
      0, __float_as_int(rule_word<MODE>(r)), kRowNewBcast + N, 0xF, 0xF, false)));
}

// max(m, |a|, |b|), one instruction (written with fmaxf each operand is first
// made a quiet number by one of its own).
__device__ __forceinline__ float max3abs(float m, float a, float b) {
  float r;
  asm("v_max3_f32 %0, %1, |%2|, |%3|" : "=v"(r) : "v"(m), "v"(a), "v"(b));
  return r;
}

struct BwShared {
  float colmax[8][2][128];
  float colmul[2][128];  // a column's multiplier (16-byte aligned)
  uint8_t tile[2][128 * 128];
};

// Group of tokens tb: its first row mb and its number of rows `live`.
template <int MODE, int ACT, bool EXPERTS>
__device__ __forceinline__ void gated_backward(
    const uint16_t* dh, const uint16_t* gu, int64_t M, int64_t F, uint8_t* q, float* s, uint8_t* qt,
    float* st, int64_t Mp, int fb, int64_t tb, int64_t mb, int live, BwShared& sh) {
  const int t = threadIdx.x, l16 = t & 15, rq = t >> 4, wave = t >> 6;
  const int64_t f0 = (int64_t)fb * kGroup + 8 * l16;

  // Byte offsets within the block's 128 tokens; of tokens past `live` loads deliver
  // zeros and stores are dropped (they are out of the resources' range).
  const __amdgpu_buffer_rsrc_t rd = make_rsrc(dh + mb * F, live * F * 2);
  const __amdgpu_buffer_rsrc_t ry = make_rsrc(gu + mb * 2 * F, live * F * 4);
  const int fs = (int)F;
  uint4 vd[4], vg[4], vu[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * rq + i;
    const uint32_t at = (uint32_t)(r * fs + (int)f0) * 2, aty = at + (uint32_t)(r * fs) * 2;
    vd[i] = load16(rd, at);
    vg[i] = load16(ry, aty);
    vu[i] = load16(ry, aty + (uint32_t)fs * 2);
  }
  float d[2][4][8];  // dgate, dup
  // (an expert's last group may have few tokens: waves without any are spared the work)
  const bool some = !EXPERTS || 16 * __builtin_amdgcn_readfirstlane(wave) < live;
  if (some) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) gate_up_grad<ACT>(vd[i], vg[i], vu[i], j, d[0][i][j], d[1][i][j]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) d[0][i][j] = d[1][i][j] = 0.f;
  }

  if (q && some) {
    // lane l16 < 8 of a DPP row: the group of half l16/4, token 4rq + l16%4
    float amax = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < 8; j += 2) a = max3abs(a, d[h][i][j], d[h][i][j + 1]);
        a = row16_max(a);
        amax = l16 == 4 * h + i ? a : amax;
      }
    const GroupRule mine = group_rule<MODE>(amax);
    const __amdgpu_buffer_rsrc_t rq_ = make_rsrc(q + mb * 2 * F, live * F * 2);
    const int r = 4 * rq + (l16 & 3);
    if (l16 < 8 && r < live) s[((l16 >> 2) * (F / kGroup) + fb) * M + mb + r] = mine.s;
    auto each = [&](auto hi) {  // (the lane to broadcast from is an immediate)
      constexpr int h = decltype(hi)::value / 4, i = decltype(hi)::value % 4;
      const GroupRule r = rule_of_lane<MODE, decltype(hi)::value>(mine);
      const float* v = d[h][i];
      const v2u o = {pack_e4m3x4(apply<MODE>(v[0], r), apply<MODE>(v[1], r), apply<MODE>(v[2], r),
                                 apply<MODE>(v[3], r)),
                     pack_e4m3x4(apply<MODE>(v[4], r), apply<MODE>(v[5], r), apply<MODE>(v[6], r),
                                 apply<MODE>(v[7], r))};
      __builtin_amdgcn_raw_buffer_store_b64(
          o, rq_, (uint32_t)((4 * rq + i) * 2 * fs + h * fs + (int)f0), 0, kNonTemporal);
    };
    each(std::integral_constant<int, 0>{});
    each(std::integral_constant<int, 1>{});
    each(std::integral_constant<int, 2>{});
    each(std::integral_constant<int, 3>{});
    each(std::integral_constant<int, 4>{});
    each(std::integral_constant<int, 5>{});
    each(std::integral_constant<int, 6>{});
    each(std::integral_constant<int, 7>{});
  }
  if (!qt) return;

#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float a = max3abs(max3abs(0.f, d[h][0][j], d[h][1][j]), d[h][2][j], d[h][3][j]);
      a = fmaxf(a, __shfl_xor(a, 16));
      a = fmaxf(a, __shfl_xor(a, 32));
      if ((t & 63) < 16) sh.colmax[wave][h][8 * l16 + j] = a;
    }
  __syncthreads();
  if (t < 256) {
    const int h = t >> 7, c = t & 127;
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) a = fmaxf(a, sh.colmax[w][h][c]);
    const GroupRule r = group_rule<MODE>(a);
    sh.colmul[h][c] = rule_word<MODE>(r);
    st[tb * 2 * F + h * F + (int64_t)fb * kGroup + c] = r.s;
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const v4f w0 = *reinterpret_cast<const v4f*>(&sh.colmul[h][8 * l16]);
    const v4f w1 = *reinterpret_cast<const v4f*>(&sh.colmul[h][8 * l16 + 4]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const GroupRule r = word_rule<MODE>(j < 4 ? w0[j] : w1[j - 4]);
      const uint32_t w = pack_e4m3x4(apply<MODE>(d[h][0][j], r), apply<MODE>(d[h][1][j], r),
                                     apply<MODE>(d[h][2][j], r), apply<MODE>(d[h][3][j], r));
      *reinterpret_cast<uint32_t*>(sh.tile[h] + tile_at(8 * l16 + j, rq)) = w;
    }
  }
  __syncthreads();
  // 2 x 128 features x 8 pieces of 16 tokens, 4 per lane
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int p = t + kBwThreads * u;
    const int h = p >> 10, c = (p >> 3) & 127, piece = p & 7;
    const v4u o = *reinterpret_cast<const v4u*>(sh.tile[h] + tile_at(c, 4 * piece));
    __builtin_nontemporal_store(
        o, reinterpret_cast<v4u*>(qt + (h * F + (int64_t)fb * kGroup + c) * Mp + tb * kGroup +
                                  16 * piece));
  }
}

// The tokens' form of a group that there is not: zeros.
__device__ __forceinline__ void no_tokens(int64_t F, uint8_t* qt, float* st, int64_t Mp, int fb0,
                                          int fb_end, int64_t tb) {
  const int t = threadIdx.x, n = (fb_end - fb0) * kGroup;
  for (int h = 0; h < 2; ++h) {
    const int64_t c0 = h * F + (int64_t)fb0 * kGroup;
    for (int c = t >> 3; c < n; c += kBwThreads / 8)
      __builtin_nontemporal_store(v4u{0, 0, 0, 0}, reinterpret_cast<v4u*>(
                                      qt + (c0 + c) * Mp + tb * kGroup + 16 * (t & 7)));
    for (int c = t; c < n; c += kBwThreads) st[tb * 2 * F + c0 + c] = 0.f;
  }
}

template <int MODE, int ACT, bool EXPERTS>
__global__ __launch_bounds__(kBwThreads) void gated_backward_kernel(
    const uint16_t* __restrict__ dh, const uint16_t* __restrict__ gu, int64_t M, int64_t F,
    const int32_t* __restrict__ off, int G, uint8_t* __restrict__ q, float* __restrict__ s,
    uint8_t* __restrict__ qt, float* __restrict__ st, int64_t Mp, int n_fblk, int blocks) {
  __shared__ __attribute__((aligned(16))) BwShared sh;
  if constexpr (EXPERTS) {
    const int n_chunk = (n_fblk + blocks - 1) / blocks;
    const int fb0 = (int)(blockIdx.x % n_chunk) * blocks;
    const int64_t tb = blockIdx.x / n_chunk;
    const int fb_end = fb0 + blocks < n_fblk ? fb0 + blocks : n_fblk;
    const ExpertSpan span = expert_span<true>(off, G, M, Mp / kGroup, (int)tb);
    if (invalid(span)) return;
    if (span.rows == 0) {  // past the last group: zeros
      if (qt) no_tokens(F, qt, st, Mp, fb0, fb_end, tb);
      return;
    }
    // (no barrier between blocks: the last one reads the tile, which the next one
    // writes behind two of its own)
    for (int fb = fb0; fb < fb_end; ++fb)
      gated_backward<MODE, ACT, true>(dh, gu, M, F, q, s, qt, st, Mp, fb, tb, span.first,
                                      span.rows, sh);
  } else {
    const int fb = blockIdx.x % n_fblk;
    const int64_t tb = blockIdx.x / n_fblk, mb = tb * kGroup;
    const int live = __builtin_amdgcn_readfirstlane(M - mb < kGroup ? (int)(M - mb) : kGroup);
    gated_backward<MODE, ACT, false>(dh, gu, M, F, q, s, qt, st, Mp, fb, tb, mb, live, sh);
  }
}

// ---- few groups: each form by workgroups of its own, in small pieces

// Rows' form of 16 tokens x 128 features: lane (t/16, t%16) owns token t/16 at
// features 8 (t%16) .. +7.  Rows past `end` are left out.
template <int MODE, int ACT>
__device__ __forceinline__ void backward_rows(const uint16_t* dh, const uint16_t* gu, int64_t M,
                                              int64_t end, int64_t F, uint8_t* q, float* s,
                                              int64_t tb, int fb) {
  const int t = threadIdx.x, l16 = t & 15, row = t >> 4;
  const int64_t mb = tb * kRowsTokens;
  if (mb >= end) return;
  const int live =
      __builtin_amdgcn_readfirstlane(end - mb < kRowsTokens ? (int)(end - mb) : kRowsTokens);
  const int fs = (int)F, f0 = fb * kGroup + 8 * l16;
  const __amdgpu_buffer_rsrc_t rd = make_rsrc(dh + mb * F, live * F * 2);
  const __amdgpu_buffer_rsrc_t ry = make_rsrc(gu + mb * 2 * F, live * F * 4);
  const uint32_t at = (uint32_t)(row * fs + f0) * 2, aty = at + (uint32_t)(row * fs) * 2;
  const uint4 vd = load16(rd, at), vg = load16(ry, aty), vu = load16(ry, aty + (uint32_t)fs * 2);
  float d[2][8], amax[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 8; ++j) gate_up_grad<ACT>(vd, vg, vu, j, d[0][j], d[1][j]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) amax[h] = max3abs(amax[h], d[h][j], d[h][j + 1]);
    amax[h] = row16_max(amax[h]);
  }
  const GroupRule mine = group_rule<MODE>(l16 == 0 ? amax[0] : amax[1]);
  if (l16 < 2 && row < live) s[(l16 * (F / kGroup) + fb) * M + mb + row] = mine.s;
  const __amdgpu_buffer_rsrc_t rq = make_rsrc(q + mb * 2 * F, live * F * 2);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const GroupRule r = h == 0 ? rule_of_lane<MODE, 0>(mine) : rule_of_lane<MODE, 1>(mine);
    const float* v = d[h];
    const v2u o = {pack_e4m3x4(apply<MODE>(v[0], r), apply<MODE>(v[1], r), apply<MODE>(v[2], r),
                               apply<MODE>(v[3], r)),
                   pack_e4m3x4(apply<MODE>(v[4], r), apply<MODE>(v[5], r), apply<MODE>(v[6], r),
                               apply<MODE>(v[7], r))};
    __builtin_amdgcn_raw_buffer_store_b64(o, rq, (uint32_t)(row * 2 * fs + h * fs + f0), 0, 0);
  }
}

struct TokensShared {
  float colmax[4][2][kTokensFeatures];
  float colmul[2][kTokensFeatures];
  uint8_t tile[2][kTokensFeatures * 128];
};

// Tokens' form of 128 tokens x 32 features: lane (t/8, t%8) owns tokens
// 4 (t/8) .. +3 at features 4 (t%8) .. +3.
template <int MODE, int ACT>
__device__ __forceinline__ void backward_tokens(const uint16_t* dh, const uint16_t* gu, int64_t mb,
                                                int live, int64_t F, uint8_t* qt, float* st,
                                                int64_t Mp, int64_t tb, int fb, TokensShared& sh) {
  const int t = threadIdx.x, l8 = t & 7, rq = t >> 3, wave = t >> 6;
  const int fs = (int)F, f0 = fb * kTokensFeatures;
  const __amdgpu_buffer_rsrc_t rd = make_rsrc(dh + mb * F, live * F * 2);
  const __amdgpu_buffer_rsrc_t ry = make_rsrc(gu + mb * 2 * F, live * F * 4);
  uint4 vd[4], vg[4], vu[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * rq + i;
    const uint32_t at = (uint32_t)(r * fs + f0 + 4 * l8) * 2, aty = at + (uint32_t)(r * fs) * 2;
    vd[i] = load8(rd, at);
    vg[i] = load8(ry, aty);
    vu[i] = load8(ry, aty + (uint32_t)fs * 2);
  }
  float d[2][4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) gate_up_grad<ACT>(vd[i], vg[i], vu[i], j, d[0][i][j], d[1][i][j]);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a = max3abs(max3abs(0.f, d[h][0][j], d[h][1][j]), d[h][2][j], d[h][3][j]);
      a = fmaxf(a, __shfl_xor(a, 8));
      a = fmaxf(a, __shfl_xor(a, 16));
      a = fmaxf(a, __shfl_xor(a, 32));
      if ((t & 63) < 8) sh.colmax[wave][h][4 * l8 + j] = a;
    }
  __syncthreads();
  if (t < 2 * kTokensFeatures) {
    const int h = t / kTokensFeatures, c = t % kTokensFeatures;
    const float a = fmaxf(fmaxf(sh.colmax[0][h][c], sh.colmax[1][h][c]),
                          fmaxf(sh.colmax[2][h][c], sh.colmax[3][h][c]));
    const GroupRule r = group_rule<MODE>(a);
    sh.colmul[h][c] = rule_word<MODE>(r);
    st[tb * 2 * F + h * F + f0 + c] = r.s;
  }
  __syncthreads();
  auto at = [](int c, int w) { return c * 128 + (((w >> 2) ^ (c >> 2)) & 7) * 16 + (w & 3) * 4; };
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const GroupRule r = word_rule<MODE>(sh.colmul[h][4 * l8 + j]);
      *reinterpret_cast<uint32_t*>(sh.tile[h] + at(4 * l8 + j, rq)) =
          pack_e4m3x4(apply<MODE>(d[h][0][j], r), apply<MODE>(d[h][1][j], r),
                      apply<MODE>(d[h][2][j], r), apply<MODE>(d[h][3][j], r));
    }
  __syncthreads();
  const int c = t >> 3, piece = t & 7;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *reinterpret_cast<v4u*>(qt + (h * F + f0 + c) * Mp + tb * kGroup + 16 * piece) =
        *reinterpret_cast<const v4u*>(sh.tile[h] + at(c, 4 * piece));
}

// The first n_rows workgroups take the rows' form, the others the tokens'.
template <int MODE, int ACT, bool EXPERTS>
__global__ __launch_bounds__(kSmallThreads) void gated_backward_small_kernel(
    const uint16_t* __restrict__ dh, const uint16_t* __restrict__ gu, int64_t M, int64_t F,
    const int32_t* __restrict__ off, int G, uint8_t* __restrict__ q, float* __restrict__ s,
    uint8_t* __restrict__ qt, float* __restrict__ st, int64_t Mp, int n_fblk, int n_rows) {
  __shared__ __attribute__((aligned(16))) TokensShared sh;
  const int b = blockIdx.x;
  const int n = n_fblk * (kGroup / kTokensFeatures), c = b - n_rows;
  const int64_t tb = b < n_rows ? b / n_fblk : c / n;
  int64_t mb = tb * kGroup, end = M;
  int live = __builtin_amdgcn_readfirstlane(M - mb < kGroup ? (int)(M - mb) : kGroup);
  if constexpr (EXPERTS) {
    const ExpertSpan span = expert_span<true>(off, G, M, Mp / kGroup, (int)tb);
    if (invalid(span)) return;
    mb = span.first;
    live = span.rows;
    end = off[G];
  }
  if (b < n_rows)
    backward_rows<MODE, ACT>(dh, gu, M, end, F, q, s, tb, b % n_fblk);
  else
    backward_tokens<MODE, ACT>(dh, gu, mb, live, F, qt, st, Mp, tb, c % n, sh);
}

// off NULL: the dense call.
template <bool EXPERTS>
static hipError_t launch(const void* dh, const void* gu, int64_t M, const int32_t* off, int G,
                         int64_t F, int act, int mode, uint8_t* q, float* s, uint8_t* qt,
                         float* st, hipStream_t stream) {
  const int64_t n_fblk = F / kGroup;
  const int64_t tb = EXPERTS ? expert_groups_most(M, G) : (M + kGroup - 1) / kGroup;
  if (n_fblk * tb > max_blocks(kBwThreads)) return hipErrorInvalidValue;
  if (n_fblk * tb <= kSmallBlocks) {
    const int64_t n_rows = q ? (M + kRowsTokens - 1) / kRowsTokens * n_fblk : 0;
    const int64_t n = n_rows + (qt ? tb * n_fblk * (kGroup / kTokensFeatures) : 0);
    auto kern = act == kActSilu
                    ? (mode == 0 ? gated_backward_small_kernel<0, kActSilu, EXPERTS>
                                 : gated_backward_small_kernel<1, kActSilu, EXPERTS>)
                    : (mode == 0 ? gated_backward_small_kernel<0, kActGeluTanh, EXPERTS>
                                 : gated_backward_small_kernel<1, kActGeluTanh, EXPERTS>);
    hipLaunchKernelGGL(kern, dim3((unsigned)n), dim3(kSmallThreads), 0, stream,
                       static_cast<const uint16_t*>(dh), static_cast<const uint16_t*>(gu), M, F,
                       off, G, q, s, qt, st, tb * kGroup, (int)n_fblk, (int)n_rows);
    return hipGetLastError();
  }
  auto kern = act == kActSilu ? (mode == 0 ? gated_backward_kernel<0, kActSilu, EXPERTS>
                                           : gated_backward_kernel<1, kActSilu, EXPERTS>)
                              : (mode == 0 ? gated_backward_kernel<0, kActGeluTanh, EXPERTS>
                                           : gated_backward_kernel<1, kActGeluTanh, EXPERTS>);
  int64_t blocks = EXPERTS ? n_fblk * tb / kBwWorkgroups : 1;
  blocks = blocks < 1 ? 1 : blocks > kBwBlocks ? kBwBlocks : blocks;
  const int64_t n_chunk = (n_fblk + blocks - 1) / blocks;
  hipLaunchKernelGGL(kern, dim3((unsigned)(n_chunk * tb)), dim3(kBwThreads), 0, stream,
                     static_cast<const uint16_t*>(dh), static_cast<const uint16_t*>(gu), M, F, off,
                     G, q, s, qt, st, tb * kGroup, (int)n_fblk, (int)blocks);
  return hipGetLastError();
}

hipError_t launch_gated_backward(const void* dh, const void* gu, int64_t M, int64_t F, int act,
                                 int mode, uint8_t* q, float* s, uint8_t* qt, float* st,
                                 hipStream_t stream) {
  return launch<false>(dh, gu, M, nullptr, 0, F, act, mode, q, s, qt, st, stream);
}

hipError_t launch_grouped_gated_backward(const void* dh, const void* gu, int64_t M,
                                         const int32_t* off, int G, int64_t F, int act, int mode,
                                         uint8_t* q, float* s, uint8_t* qt, float* st,
                                         hipStream_t stream) {
  return launch<true>(dh, gu, M, off, G, F, act, mode, q, s, qt, st, stream);
}

#ifdef FP8Q_DEBUG_CHECKS
hipError_t backward_offsets_error_take(hipStream_t stream, int* flag) {
  return take_experts_error(stream, flag);
}
#endif

}  // namespace fp8q
