/*
 * fp8q.h -- C ABI of the MI355X (gfx950) fine-grained block-scaled FP8 library.
 *
 * The method (pages cited by site and passage; they carry no section numbers):
 *   - the-good.kr free board post 2169793, fine-grained quantization passage:
 *     the max-abs is computed online for every 1x128 activation tile and every
 *     128x128 weight block, the scaling factor is derived from it, and the
 *     values are cast to FP8 online; E4M3 (4-bit exponent, 3-bit mantissa) is
 *     used for all tensors (mixed-precision framework passage).
 *   - why-be.co.kr as_center post 57820, promotion passage: once an interval
 *     of N_C elements along K is reached, the partial results are moved out of
 *     the matrix unit, multiplied by the scaling factors and added into FP32
 *     registers; pkd.ac.th webboard post 78017 (increased-precision
 *     accumulation passage) fixes N_C = 128.
 *   - why-be.co.kr as_center post 57820 / pkd.ac.th webboard post 78017,
 *     inference-deployment passages: per-expert GEMMs over small token batches
 *     (routed top-8 of 256 experts), memory-bound in decoding.
 *   - the-good.kr free board post 2169793, mixed-precision framework passage:
 *     the forward GEMM and both backward GEMMs of a linear layer run in FP8
 *     (fp8q_quantize_act_t, fp8q_quantize_weight_t, fp8q_gemm_rowscaled), said
 *     to double their speed in theory over BF16 (fp8q_gemm_bf16 is the BF16
 *     GEMM of the same kernel family that claim is measured against).
 *
 * Conventions for every call:
 *   - Every data pointer is a DEVICE pointer on the current HIP device.  The
 *     caller allocates and frees all memory; the library allocates nothing (but
 *     host memory during a call: fp8q_adamw, to sort more than 64 tensors),
 *     keeps no pointer after returning, creates no stream and never
 *     synchronizes.  Work is enqueued on `stream` (NULL = the default stream)
 *     and runs asynchronously.
 *   - Layouts are packed, row-major, with no stride arguments.
 *   - Arguments are validated on the host before any device call, in this
 *     order: NULL pointers (a pointer may be NULL only when its extent is 0),
 *     shapes, alignment, enums, then the current device must be gfx950.  A
 *     validation error returns without side effects.  A launch failure
 *     returns FP8Q_ERR_LAUNCH; output contents are then undefined.
 *   - Inputs must be finite; outputs must not alias inputs.
 *   - E4M3 here is the OCP "E4M3FN" encoding (bias 7, no infinities, max 448).
 *   - Thread-safe; the only global state is a per-device architecture cache
 *     (and, in FP8Q_DEBUG_CHECKS builds, a per-device offsets-error flag:
 *     grouped calls on one device that overlap in time share it, so one of
 *     them may report the other's invalid offsets).
 */
#ifndef FP8Q_H
#define FP8Q_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP8Q_ABI_VERSION 3

typedef enum {
  FP8Q_OK = 0,
  FP8Q_ERR_NULL = 1,        /* a required pointer is NULL                      */
  FP8Q_ERR_SHAPE = 2,       /* negative size, or K / N not a multiple of 128,
                               or G < 1                                          */
  FP8Q_ERR_ALIGN = 3,       /* data pointer not 16-byte aligned, or scale /
                               offset pointer not 4-byte aligned                 */
  FP8Q_ERR_ENUM = 4,        /* unknown scale mode or output dtype              */
  FP8Q_ERR_DEVICE = 5,      /* no current HIP device, or it is not gfx950      */
  FP8Q_ERR_LAUNCH = 6,      /* the kernel launch failed, or would need more
                               than its 2^32 lanes                              */
  FP8Q_ERR_UNSUPPORTED = 7, /* valid request the library does not implement   */
  FP8Q_ERR_OFFSETS = 8      /* grouped calls, FP8Q_DEBUG_CHECKS builds only: the
                               device offsets are not 0 = off[0] <= ... <=
                               off[G] <= M_total                                  */
} fp8q_status;

typedef enum {
  /* s = fl32(amax / 448); codes = E4M3_RNE(fl32(x * fl32(448 / amax))).
     A group whose 448/amax is not finite (amax == 0 or below 448/FLT_MAX)
     is flushed: s = 0 and every code is a signed zero (0x00 / 0x80).      */
  FP8Q_SCALE_F32 = 0,
  /* s = 2^e, e the smallest integer with 448 * 2^e >= amax (why-be.co.kr
     as_center post 72410: scaling factors that are integral powers of 2);
     codes = E4M3_RNE(x * 2^-e).  amax == 0 gives s = 0 and signed zeros. */
  FP8Q_SCALE_POW2 = 1
} fp8q_scale_mode;

typedef enum {
  FP8Q_OUT_F32 = 0,   /* C stored as float32                              */
  FP8Q_OUT_BF16 = 1   /* C stored as bfloat16, round-to-nearest-even of
                         the FP32 accumulator                             */
} fp8q_out_dtype;

/*
 * 1x128 activation quantization (fine-grained quantization passage of the
 * the-good.kr post: one scale per activation row and 128 consecutive K).
 *   x_bf16 : [M][K] bfloat16, row-major; 16-byte aligned.
 *   q      : [M][K] uint8 E4M3 codes (output); 16-byte aligned.
 *   s      : [K/128][M] float32 scales (output), group-major so that the M
 *            scales of one K group are contiguous; 4-byte aligned.
 *   M >= 0 (M == 0 is a no-op), K >= 0 with K % 128 == 0.
 * Results are bit-exact functions of the input (no reduction-order effects).
 */
fp8q_status fp8q_quantize_act(const void* x_bf16, int64_t M, int64_t K,
                              uint8_t* q, float* s, fp8q_scale_mode mode,
                              hipStream_t stream);

/*
 * 128x128 weight-block quantization (same passage: one scale per block of
 * 128 rows of N by 128 columns of K).
 *   w_bf16 : [N][K] bfloat16, row-major; 16-byte aligned.
 *   q      : [N][K] uint8 E4M3 codes (output); 16-byte aligned.
 *   s      : [N/128][K/128] float32 scales, row-major (output).
 *   N % 128 == 0, K % 128 == 0.  A stack of G experts' weights [G][N][K]
 *   may be passed as one [G*N][K] matrix: blocks never straddle experts, and
 *   the scales come out as [G][N/128][K/128].
 */
fp8q_status fp8q_quantize_weight(const void* w_bf16, int64_t N, int64_t K,
                                 uint8_t* q, float* s, fp8q_scale_mode mode,
                                 hipStream_t stream);

/*
 * Block-scaled FP8 GEMM with promotion every 128 K (promotion passage of the
 * why-be.co.kr post 57820, interval from the pkd.ac.th post):
 *   C[m][n] = sum_g (a_s[g][m] * w_s[n/128][g]) * P_g[m][n],
 *   P_g[m][n] = sum_{k in [128g, 128g+128)} dec(a_q[m][k]) * dec(w_q[n][k]);
 * each P_g is formed by the matrix cores from a zero start and folded into
 * the FP32 accumulator by a fused multiply-add on the vector ALUs.
 *   a_q : [M][K] uint8, a_s : [K/128][M] float32  (from fp8q_quantize_act)
 *   w_q : [N][K] uint8, w_s : [N/128][K/128] float32 (from fp8q_quantize_weight)
 *   c   : [M][N] float32 or bfloat16 (per `out`), row-major (output).
 *   M >= 0, N % 128 == 0, K % 128 == 0.
 * FP8Q_ERR_UNSUPPORTED: K == 0 with M*N > 0 (C would be all zeros), K > 2^22,
 *   or M * (K/128) * 4 >= 2^31 (32-bit load offsets).
 * ACCURACY (FP8 matrix cores).  Within each P_g the gfx950 FP8 instruction
 * takes the products in groups of 8 consecutive K; with E the largest
 * exponent sum ex(a) + ex(w) of a group's non-zero products (ex = unbiased
 * E4M3 exponent, -6 for subnormals), it truncates every product toward zero
 * to a multiple of 2^(E-13), sums the group exactly, and adds the group sums
 * in FP32 (a measured property of the hardware, the analogue of the 14-bit
 * fixed-point accumulation the why-be.co.kr post 72410 describes for Hopper).
 * A product p of exponent sum e is a multiple of 2^(e-6), so it is kept
 * exactly when e >= E-7.  Hence, per output, from the operands alone:
 *   |C - C_exact| <= T + (G + 20) * 2^-24 * S   (+ half a BF16 ulp of C_exact
 *                                                for BF16 output), where
 *   S = sum_k |dec(a_q[m][k]) * s_a| * |dec(w_q[n][k]) * s_w|,
 *   T = sum_g |s_a * s_w| * sum_{8-K groups of chunk g}
 *           sum_{k in group, e_k < E-7} min(|p_k|, 2^(E-13)),
 *   G = K/128 (the FP32 additions inside the instruction, the rounding of
 *   s_a * s_w and of the promotion per chunk).  T is what the matrix core
 * can lose; it can exceed the 1e-5 * S tolerance where one product dominates
 * an 8-K group (an outlier channel).  fp8q_gemm_precise meets the tolerance.
 * RANGE (both modes): the bounds assume every product s_a * s_w is a normal
 * FP32 number (>= 2^-126) and no partial sum overflows; outside that range
 * the FP32 arithmetic of the promotion itself loses precision (a subnormal
 * s_a * s_w keeps fewer significant bits).
 */
fp8q_status fp8q_gemm(const uint8_t* a_q, const float* a_s,
                      const uint8_t* w_q, const float* w_s,
                      int64_t M, int64_t N, int64_t K,
                      void* c, fp8q_out_dtype out, hipStream_t stream);

/*
 * Precise mode of fp8q_gemm: the same operands, layouts, arguments, errors
 * and promotion every 128 K, with each chunk partial P_g formed from the E4M3
 * codes widened exactly to FP16 (every E4M3 value is an FP16 value) by FP16
 * matrix-core instructions, whose accumulation is far wider than the FP8
 * instruction's 14-bit step (the higher-precision accumulation the
 * why-be.co.kr post 57820 asks for in its hardware-suggestion passage).  Half
 * the matrix-core rate of fp8q_gemm.
 * PRECISE ACCURACY.  Measured on gfx950, the FP16 instruction sums groups of
 * 8 consecutive products aligned to the group's largest exponent with a
 * window of about 25 bits and adds the group sums to its C input in FP32; a
 * chunk partial (4 instructions) is within 32 * 2^-24 * sum_chunk |p| of the
 * exact one.  Hence, per output, with S and G as for fp8q_gemm:
 *   |C - C_exact| <= (G + 34) * 2^-24 * S  (+ half a BF16 ulp of C_exact),
 * which is within the 1e-5 * S tolerance for K <= 17024 (G <= 133); on
 * random data the error stays near 1e-7 * S at any K (8192 x 8192 x 65536
 * measured: 1.4e-8 * S).  The RANGE clause of fp8q_gemm applies.
 */
fp8q_status fp8q_gemm_precise(const uint8_t* a_q, const float* a_s,
                              const uint8_t* w_q, const float* w_s,
                              int64_t M, int64_t N, int64_t K,
                              void* c, fp8q_out_dtype out, hipStream_t stream);

/*
 * fp8q_gemm with the group scales applied by the matrix core ("MMA with
 * group scaling", the hardware-suggestion passage of the why-be.co.kr post
 * 57820; power-of-two scaling factors, the inference passage of post 72410):
 * each chunk's block-scaled FP8 MFMA takes s_a and s_w as E8M0 exponent
 * bytes, so P_g comes out of the matrix core already scaled, from a zero
 * start, and the promotion adds it into the FP32 accumulators.  The same
 * operands, layouts, arguments and errors as fp8q_gemm, for scales that are
 * powers of two or zero (FP8Q_SCALE_POW2 quantizers).  A scale below 2^-126,
 * which E8M0 cannot hold next to the others, is split exactly between the
 * matrix core (2^-127) and the promotion.
 * RESULT: within the RANGE clause of fp8q_gemm, bitwise equal to fp8q_gemm on
 * the same power-of-two-scaled operands (a power-of-two scaling commutes with
 * the matrix core's truncation and with FP32 rounding), hence the same
 * ACCURACY clause.  Scales that are not powers of two are used as
 * 2^floor(log2 s): their fraction bits are ignored.
 * The matrix core's C input cannot carry the running sum instead: it joins
 * the 14-bit alignment of the products, so each chunk starts from zero.
 */
fp8q_status fp8q_gemm_mfma_scaled(const uint8_t* a_q, const float* a_s,
                                  const uint8_t* w_q, const float* w_s,
                                  int64_t M, int64_t N, int64_t K,
                                  void* c, fp8q_out_dtype out, hipStream_t stream);

/*
 * Grouped (per-expert) variant.  Rows [off[e], off[e+1]) of a_q use expert
 * e's weights w_q + e*N*K and scales w_s + e*(N/128)*(K/128).
 *   a_q : [M_total][K] uint8, a_s : [K/128][M_total] float32.
 *   off : DEVICE int32[G+1] with 0 = off[0] <= off[1] <= ... <= off[G] <=
 *         M_total; experts with no rows are allowed.  The kernel checks this
 *         on the device before any memory access: with invalid offsets the
 *         launch writes nothing (c keeps its contents) and, since the check
 *         runs on the device, the call still returns FP8Q_OK; a library built
 *         with FP8Q_DEBUG_CHECKS (fp8q_debug_checks() == 1) synchronizes the
 *         stream after each grouped launch and returns FP8Q_ERR_OFFSETS.
 *   w_q : [G][N][K] uint8, w_s : [G][N/128][K/128] float32.
 *   c   : [M_total][N] (output); rows >= off[G] are left untouched.
 *   G >= 1, N % 128 == 0, K % 128 == 0.  No host synchronization is needed
 *   between the producer of `off` and this call.
 * FP8Q_ERR_UNSUPPORTED: G > 1024, or the dense call's K / row-count limits
 *   with M_total in place of M.  Accuracy as for fp8q_gemm.
 */
fp8q_status fp8q_grouped_gemm(const uint8_t* a_q, const float* a_s, int64_t M_total,
                              const int32_t* off, int32_t G,
                              const uint8_t* w_q, const float* w_s,
                              int64_t N, int64_t K,
                              void* c, fp8q_out_dtype out, hipStream_t stream);

/* Precise mode of fp8q_grouped_gemm (chunk partials as in fp8q_gemm_precise);
   everything else as fp8q_grouped_gemm. */
fp8q_status fp8q_grouped_gemm_precise(const uint8_t* a_q, const float* a_s, int64_t M_total,
                                      const int32_t* off, int32_t G,
                                      const uint8_t* w_q, const float* w_s,
                                      int64_t N, int64_t K,
                                      void* c, fp8q_out_dtype out, hipStream_t stream);

/*
 * Backward GEMMs (the-good.kr post 2169793, mixed-precision framework
 * passage: Fprop, Dgrad and Wgrad of a linear layer all run in FP8; scales
 * are per group along each GEMM's inner dimension).  For Y = X W^T:
 *   Dgrad  dX = dY W     : fp8q_gemm(fp8q_quantize_act(dY), fp8q_quantize_weight_t(W))
 *   Wgrad  dW = dY^T X   : fp8q_gemm_rowscaled(fp8q_quantize_act_t(dY), fp8q_quantize_act_t(X))
 *
 * Transposed activation quantization: groups of 128 consecutive rows (tokens)
 * of one column, the 1x128 rule of fp8q_quantize_act applied to x^T.
 *   x_bf16 : [M][K] bfloat16, row-major; 16-byte aligned.
 *   q_t    : [K][M] uint8 E4M3 codes of x^T (output); 16-byte aligned.
 *   s_t    : [M/128][K] float32 (output): s_t[g][k] scales rows 128g..128g+127
 *            of column k (the activation-scale layout of an operand with K rows).
 *   M % 128 == 0, K % 128 == 0.
 */
fp8q_status fp8q_quantize_act_t(const void* x_bf16, int64_t M, int64_t K,
                                uint8_t* q_t, float* s_t, fp8q_scale_mode mode,
                                hipStream_t stream);

/*
 * Transposed weight quantization: the 128x128 blocks of fp8q_quantize_weight
 * with their codes written transposed, i.e. the weight operand W^T of Dgrad.
 *   w_bf16 : [N][K] bfloat16, row-major; 16-byte aligned.
 *   q_t    : [K][N] uint8 E4M3 codes of w^T (output); 16-byte aligned.
 *   s_t    : [K/128][N/128] float32 (output; the transpose of the block scales).
 *   N % 128 == 0, K % 128 == 0.
 */
fp8q_status fp8q_quantize_weight_t(const void* w_bf16, int64_t N, int64_t K,
                                   uint8_t* q_t, float* s_t, fp8q_scale_mode mode,
                                   hipStream_t stream);

/*
 * Block-scaled FP8 GEMM whose both operands carry 1x128 row-group scales
 * (the weight-gradient GEMM; promotion every 128 K as in fp8q_gemm):
 *   C[m][n] = sum_g (a_s[g][m] * b_s[g][n]) * P_g[m][n]
 *   a_q : [M][K] uint8, a_s : [K/128][M] float32;
 *   b_q : [N][K] uint8, b_s : [K/128][N] float32 (both as from fp8q_quantize_act
 *         or fp8q_quantize_act_t);
 *   c   : [M][N] float32 or bfloat16 (per `out`), row-major (output).
 *   M >= 0, N % 128 == 0, K % 128 == 0.
 * FP8Q_ERR_UNSUPPORTED: as fp8q_gemm, with the row-count limit applied to
 *   both M and N.  Accuracy: the ACCURACY clause of fp8q_gemm with
 *   b_s[g][n] in place of w_s[n/128][g].
 */
fp8q_status fp8q_gemm_rowscaled(const uint8_t* a_q, const float* a_s,
                                const uint8_t* b_q, const float* b_s,
                                int64_t M, int64_t N, int64_t K,
                                void* c, fp8q_out_dtype out, hipStream_t stream);

/* Precise mode of fp8q_gemm_rowscaled (chunk partials as in
   fp8q_gemm_precise); everything else as fp8q_gemm_rowscaled. */
fp8q_status fp8q_gemm_rowscaled_precise(const uint8_t* a_q, const float* a_s,
                                        const uint8_t* b_q, const float* b_s,
                                        int64_t M, int64_t N, int64_t K,
                                        void* c, fp8q_out_dtype out, hipStream_t stream);

/*
 * BF16 GEMM of the same kernel family, without quantization: the reference
 * point for the FP8 path's speed (the-good.kr post 2169793, mixed-precision
 * framework passage: running the GEMMs in FP8 is said to double their speed
 * in theory over BF16) and accuracy.
 *   C[m][n] = sum_k a[m][k] * w[n][k]
 *   a : [M][K] bfloat16, w : [N][K] bfloat16, row-major; 16-byte aligned.
 *   c : [M][N] float32 or bfloat16 (per `out`), row-major (output).
 *   M >= 0, N % 128 == 0, K % 128 == 0 (the shape rules of fp8q_gemm).
 * FP8Q_ERR_UNSUPPORTED: K == 0 with M*N > 0, or K > 2^21 (32-bit load
 *   offsets over rows of 2K bytes).
 * Accuracy: the products of BF16 values are exact in FP32; the matrix core
 * accumulates them (32 per instruction, with the running sum as its C input)
 * to FP32 accuracy, so |C - C_exact| <= 1e-5 * sum_k |a[m][k]| * |w[n][k]|
 * (plus half a BF16 ulp for BF16 output).
 */
fp8q_status fp8q_gemm_bf16(const void* a, const void* w, int64_t M, int64_t N, int64_t K,
                           void* c, fp8q_out_dtype out, hipStream_t stream);

/*
 * GEMMs that quantize their BF16 activation operand themselves: the FP8 cast
 * fused with the transfer of the activations into on-chip memory, instead of
 * writing the codes to HBM and reading them back (why-be.co.kr as_center post
 * 57820, hardware-suggestion passage; the-good.kr post 2169793, fine-grained
 * quantization passage).  Every K chunk of a tile's activation rows is
 * quantized by the rule of fp8q_quantize_act with scale mode `mode`, so, for
 * finite inputs (the contract of every call),
 *   fp8q_gemm_fused(x, w_q, w_s, ...) == fp8q_gemm(fp8q_quantize_act(x, mode), w_q, w_s, ...)
 * bit for bit, and likewise the grouped call against fp8q_grouped_gemm.  The
 * codes and scales of x are not written out.  Each tile re-quantizes its rows
 * (once per 256 output columns).
 *   x_bf16 : [M][K] (or [M_total][K]) bfloat16, row-major; 16-byte aligned.
 *   w_q, w_s, off, c, out and the shape rules: as fp8q_gemm / fp8q_grouped_gemm.
 * FP8Q_ERR_UNSUPPORTED: K == 0 with output rows, K > 2^21 (32-bit load
 *   offsets over rows of 2K bytes), or (grouped) G > 1024.
 * Accuracy as fp8q_gemm (the same arithmetic on the same codes).
 */
fp8q_status fp8q_gemm_fused(const void* x_bf16, const uint8_t* w_q, const float* w_s,
                            int64_t M, int64_t N, int64_t K,
                            void* c, fp8q_out_dtype out, fp8q_scale_mode mode,
                            hipStream_t stream);

fp8q_status fp8q_grouped_gemm_fused(const void* x_bf16, int64_t M_total,
                                    const int32_t* off, int32_t G,
                                    const uint8_t* w_q, const float* w_s,
                                    int64_t N, int64_t K,
                                    void* c, fp8q_out_dtype out, fp8q_scale_mode mode,
                                    hipStream_t stream);

/*
 * The feed-forward layer in 8 bits (the calls below): products of int8 codes
 * with one scale per token and per output channel, the gated block
 * act(gate) * up on int8 and on block-scaled E4M3 operands, and the backward
 * pass of its activation.
 */
typedef enum {
  FP8Q_ACT_SILU = 0,      /* act(x) = x / (1 + exp(-x))                                  */
  FP8Q_ACT_GELU_TANH = 1  /* act(x) = x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3)))      */
} fp8q_activation;

/*
 * Per-token symmetric int8 quantization (per output channel for a weight
 * matrix [N][K]):
 *   s[m] = fl32(amax_m / 127),
 *   q[m][k] = rne(fl32(x[m][k] * inv_m)), inv_m = fl32(127 * fl32(1 / amax_m)).
 * A row whose inv is not finite (amax 0 or below 127/FLT_MAX) is flushed: s = 0
 * and every code 0.
 *   x_bf16 : [M][K] bfloat16, row-major; 16-byte aligned.
 *   q      : [M][Kp] int8 codes in [-127, 127] (output), Kp = K rounded up to a
 *            multiple of 16, zeros past K; 16-byte aligned.
 *   s      : [M] float32 (output); 4-byte aligned.
 *   M >= 0 (M == 0 is a no-op), any K >= 1 (K == 0 with M > 0: FP8Q_ERR_UNSUPPORTED).
 * Results are bit-exact functions of the input.
 */
fp8q_status fp8q_quantize_token_i8(const void* x_bf16, int64_t M, int64_t K, int8_t* q, float* s,
                                   hipStream_t stream);

/*
 * int8 product with scales per token and per channel:
 *   C[m][n] = (sum_k a_q[m][k] * w_q[n][k]) * a_s[m] * w_s[n] + bias[n].
 *   a_q : [M][K] int8, a_s : [M] float32; w_q : [N][K] int8, w_s : [N] float32
 *         (as from fp8q_quantize_token_i8; the code -128 is allowed too)
 *   bias: [N] float32, or NULL for none; 4-byte aligned.
 *   c   : [M][N] float32 or bfloat16 (per `out`), row-major (output).
 *   M >= 0, any N >= 0, K % 16 == 0.
 * FP8Q_ERR_UNSUPPORTED: K == 0 with M*N > 0, or K >= 131072 (the sum could
 *   leave int32).
 * Accuracy: the integer sum is exact; it is converted to FP32 and scaled by
 * two FP32 products (and one addition), so
 *   |C - C_exact| <= 4 * 2^-24 * (|C_exact - bias| + |bias|)  (+ half a BF16 ulp).
 * RANGE: the bound assumes that sum * a_s[m], formed first, and its product with
 * w_s[n] are normal FP32 numbers or 0 (no overflow, nothing below 2^-126).
 */
fp8q_status fp8q_gemm_i8(const int8_t* a_q, const float* a_s, const int8_t* w_q, const float* w_s,
                         const float* bias, int64_t M, int64_t N, int64_t K, void* c,
                         fp8q_out_dtype out, hipStream_t stream);

/*
 * Gated block on int8 operands: with Y = fp8q_gemm_i8's product (no bias) of
 * the stacked gate and up weights,
 *   h[m][f] = act(Y[m][f]) * Y[m][F + f],
 * formed in FP32 from the exact integer sums; Y is not written.
 *   a_q : [M][K] int8, a_s : [M] float32;
 *   w_q : [2F][K] int8 (rows 0..F-1 gate, F..2F-1 up), w_s : [2F] float32
 *   h   : [M][F] float32 or bfloat16 (per `out`) (output).
 *   M >= 0, any F >= 0, K % 16 == 0; errors and RANGE as fp8q_gemm_i8.
 * act(x) = x sigma(y) (y = x, or 2 sqrt(2/pi) (x + 0.044715 x^3)) is evaluated
 * in FP32 with an error of at most 2^-128 |x| + 2^-149 and, relative to |act(x)|,
 * 8 * 2^-24 for FP32 output, (16 + 8|y|) 2^-24 for BF16 output.
 */
fp8q_status fp8q_gemm_i8_gated(const int8_t* a_q, const float* a_s, const int8_t* w_q,
                               const float* w_s, int64_t M, int64_t F, int64_t K,
                               fp8q_activation act, void* h, fp8q_out_dtype out,
                               hipStream_t stream);

/*
 * Gated block on block-scaled E4M3 operands: with Y = fp8q_gemm's product of
 * the stacked gate and up weights (accuracy and RANGE clauses of fp8q_gemm),
 *   h[m][f] = act(Y[m][f]) * Y[m][F + f].
 * With many rows Y's sums are fp8q_gemm's bit for bit.  Few rows (always up to
 * 16) take a kernel that adds a sum's chunks as 8 partial sums: within the same
 * bound, but the last bits differ, so that a token's result depends on whether its
 * call holds few rows or many.
 *   a_q : [M][K] uint8, a_s : [K/128][M] float32 (from fp8q_quantize_act)
 *   w_q : [2F][K] uint8 (rows 0..F-1 gate, F..2F-1 up), w_s : [2F/128][K/128]
 *         float32 (from fp8q_quantize_weight)
 *   h   : [M][F] float32 or bfloat16 (per `out`) (output).
 *   gate_up : [M][2F] bfloat16 Y for the backward pass (output), or NULL;
 *         h is formed from the FP32 Y, not from this rounded copy.
 *   M >= 0, F % 128 == 0, K % 128 == 0; errors as fp8q_gemm.
 * act(x) (as above) is evaluated in FP32 with an error of at most
 * (16 + 8|y|) 2^-24 |act(x)| + 2^-128 |x| + 2^-149: the sums of the FP8 matrix
 * cores carry more.
 */
fp8q_status fp8q_gemm_gated(const uint8_t* a_q, const float* a_s, const uint8_t* w_q,
                            const float* w_s, int64_t M, int64_t F, int64_t K,
                            fp8q_activation act, void* h, fp8q_out_dtype out, void* gate_up,
                            hipStream_t stream);

/*
 * The same for routed experts: rows [off[e], off[e+1]) use expert e's weights.
 *   off : DEVICE int32[G+1], as for fp8q_grouped_gemm (validated on the device:
 *         with invalid offsets nothing is written).
 *   w_q : [G][2F][K] uint8, w_s : [G][2F/128][K/128] float32.
 *   h   : [M_total][F], gate_up : [M_total][2F] or NULL; rows >= off[G] are
 *         left untouched.
 *   Errors as fp8q_grouped_gemm.
 */
fp8q_status fp8q_grouped_gemm_gated(const uint8_t* a_q, const float* a_s, int64_t M_total,
                                    const int32_t* off, int32_t G, const uint8_t* w_q,
                                    const float* w_s, int64_t F, int64_t K, fp8q_activation act,
                                    void* h, fp8q_out_dtype out, void* gate_up,
                                    hipStream_t stream);

/*
 * Backward pass of the gated activation, quantized for both gradient GEMMs of
 * the gate/up projection in one pass over its inputs:
 *   dgate = dh * up * act'(gate), dup = dh * act(gate), dY = [dgate | dup] in
 *   FP32, then (scale rule `mode`, as fp8q_quantize_act)
 *   q, s   : dY in 1x128 groups along the features: [M][2F] codes and
 *            [2F/128][M] scales (the A operand of dX = dY W);
 *   qt, st : dY^T in groups of 128 tokens: [2F][Mp] codes and [Mp/128][2F]
 *            scales, Mp = M rounded up to a multiple of 128, codes past M zero
 *            (the A operand of dW = dY^T X, fp8q_gemm_rowscaled).
 * Either pair may be NULL: it is then not computed.
 *   dh      : [M][F] bfloat16; gate_up : [M][2F] bfloat16 (from fp8q_gemm_gated).
 *   M >= 0, F >= 0 with F % 128 == 0.
 * FP8Q_ERR_UNSUPPORTED: F > 2^22 (32-bit offsets within 128 tokens).
 * dY is not rounded before it is quantized.  With act(x) = x sigma(y), its FP32
 * values are within
 *   (16 + 8|y|) 2^-24 |dh| |up| (|act'(gate)| + |gate y' sigma(y) sigma(-y)|)  and
 *   (16 + 8|y|) 2^-24 |dh| |act(gate)|
 * of the exact dgate and dup (|y| counted up to 100, and 2^-119 beside it): the
 * terms' size is what counts, so near the zero of act' dgate's error relative to
 * itself is larger.  A code can differ from that of the exact dY where that lies
 * within this error (its own, or of its group's largest value) of a rounding
 * boundary.
 * RANGE: dY must stay below FLT_MAX.
 */
fp8q_status fp8q_gated_backward(const void* dh, const void* gate_up, int64_t M, int64_t F,
                                fp8q_activation act, fp8q_scale_mode mode, uint8_t* q, float* s,
                                uint8_t* qt, float* st, hipStream_t stream);

/*
 * The rest of a training step around the FP8 products (the calls below): layer
 * norm and its backward pass, the gradients of experts' weights, and AdamW.
 */

/*
 * Layer norm of rows: z = (x - mean) * rstd, rstd = 1 / sqrt(var + eps), var the
 * mean square of x - mean; y = z * weight + bias, in FP32 and rounded once.
 *   x      : [M][N] float32 or bfloat16 (per `x_type`), row-major; 16-byte aligned.
 *   weight : [N] float32; bias: [N] float32, or NULL for none.
 *   y      : [M][N] float32 or bfloat16 (per `y_type`) (output), or NULL.
 *   q, s   : y in 1x128 groups by the rule of fp8q_quantize_act (from y in FP32,
 *            not from its BF16 rounding): [M][N] codes, 16-byte aligned, and
 *            [N/128][M] scales (output); or both NULL.  One of y and q is wanted.
 *   mean, rstd : [M] float32 (output).
 *   M >= 0, 1 <= N <= 16384 (more: FP8Q_ERR_UNSUPPORTED); with q, N % 128 == 0.
 *   eps >= 0, finite (else FP8Q_ERR_UNSUPPORTED).
 * ACCURACY.  mean and var are FP32 sums over the row, var about the mean.  With u =
 * 2^-24 and D = 40 u mean|x|:
 *   |mean - mean_exact| <= D,  rstd within 23 u + (D rstd)^2 / 2 relative,
 *   |z - z_exact| <= rstd D + (25 u + (D rstd)^2 / 2) |z|,  and y within
 *   |weight| times that + 2 u |z weight| + u |y| (and half a BF16 ulp).
 * This holds for every eps and every row up to |x| = 2^126 of which 1 / sqrt(var + eps)
 * is a normal FP32 number (rows whose squares FP32 cannot hold are summed scaled by a
 * power of two).  With eps == 0 a constant row has rstd = infinity and z = NaN.
 */
fp8q_status fp8q_layer_norm(const void* x, fp8q_out_dtype x_type, const float* weight,
                            const float* bias, int64_t M, int64_t N, float eps, void* y,
                            fp8q_out_dtype y_type, uint8_t* q, float* s, fp8q_scale_mode mode,
                            float* mean, float* rstd, hipStream_t stream);

/*
 * Backward pass of layer norm.  With z as above and gz = dy * weight:
 *   dx = rstd * (gz - mean(gz) - z * mean(gz * z))     (means over the row),
 *   dweight[n] = sum over rows of dy * z,  dbias[n] = sum over rows of dy.
 *   dy     : [M][N] float32 or bfloat16 (per `dy_type`); x as above, mean and rstd
 *            as fp8q_layer_norm wrote them.
 *   dx     : [M][N] of x's type (output); dweight: [N] float32 (output); dbias:
 *            [N] float32 (output), or NULL.
 *   workspace : fp8q_layer_norm_backward_workspace(M, N) bytes, 16-byte aligned,
 *            whose contents do not matter before or after the call; calls that can
 *            run at the same time need one each.  NULL where that is 0.
 *   M >= 0 (with M == 0 dweight and dbias are zeros), N and x as above.
 * The sums over rows are FP32 in a fixed order: the same bits every time.
 */
int64_t fp8q_layer_norm_backward_workspace(int64_t M, int64_t N);
fp8q_status fp8q_layer_norm_backward(const void* dy, fp8q_out_dtype dy_type, const void* x,
                                     fp8q_out_dtype x_type, const float* weight,
                                     const float* mean, const float* rstd, int64_t M, int64_t N,
                                     void* dx, float* dweight, float* dbias, void* workspace,
                                     hipStream_t stream);

/*
 * Tokens by expert, transposed.  The weight gradient of expert e sums over its
 * tokens, rows [off[e], off[e+1]), so its operands carry scales in groups of 128
 * of them.  Expert e's n_e rows take ceil(n_e/128) groups, which follow those of
 * expert e-1: no group holds two experts' tokens.  An operand has
 *   T = fp8q_expert_columns(M_total, G) columns, 128 times the most groups that
 * M_total rows in G experts can take; those past an expert's last row, and past the
 * last expert, hold zero codes (groups past the last expert zero scales).
 * off is a DEVICE int32[G+1], 0 = off[0] <= ... <= off[G] <= M_total, checked on the
 * device: with invalid offsets these calls write nothing and return FP8Q_OK (debug
 * builds: FP8Q_ERR_OFFSETS), as fp8q_grouped_gemm does.  G <= 1024 (more:
 * FP8Q_ERR_UNSUPPORTED).
 */
int64_t fp8q_expert_columns(int64_t M_total, int32_t G);

/* fp8q_quantize_act_t by expert.
 *   x_bf16 : [M_total][K] bfloat16; 16-byte aligned.
 *   q_t    : [K][T] codes (output); s_t : [T/128][K] float32 (output).
 *   K % 128 == 0, K <= 2^22 (more: FP8Q_ERR_UNSUPPORTED). */
fp8q_status fp8q_grouped_quantize_act_t(const void* x_bf16, int64_t M_total, const int32_t* off,
                                        int32_t G, int64_t K, uint8_t* q_t, float* s_t,
                                        fp8q_scale_mode mode, hipStream_t stream);

/* fp8q_gated_backward by expert: qt [2F][T] and st [T/128][2F] have the groups of
 * tokens above, q and s are as there (rows past off[G] are left untouched). */
fp8q_status fp8q_grouped_gated_backward(const void* dh, const void* gate_up, int64_t M_total,
                                        const int32_t* off, int32_t G, int64_t F,
                                        fp8q_activation act, fp8q_scale_mode mode, uint8_t* q,
                                        float* s, uint8_t* qt, float* st, hipStream_t stream);

/*
 * Weight gradients of all experts: fp8q_gemm_rowscaled over each expert's groups,
 *   C[e][n][k] = sum over expert e's groups g of (a_s[g][n] * b_s[g][k]) * P_g[n][k].
 *   a_q : [N][T] uint8, a_s : [T/128][N] float32; b_q : [K][T] uint8, b_s : [T/128][K]
 *         float32 (both as from the calls above, with the same off)
 *   T   : the operands' columns, a multiple of 128, at least the groups that off
 *         asks for (fewer: invalid offsets).
 *   c   : [G][N][K] float32 or bfloat16 (per `out`) (output); zeros for an expert
 *         without rows.
 *   N % 128 == 0, K % 128 == 0.  FP8Q_ERR_UNSUPPORTED: G > 1024, T > 2^24, N or K
 *   > 2^22 (32-bit offsets).
 * Accuracy: the ACCURACY clause of fp8q_gemm over each expert's groups, and for the
 * precise call that of fp8q_gemm_precise.
 */
fp8q_status fp8q_grouped_gemm_rowscaled(const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                                        const float* b_s, int64_t T, const int32_t* off,
                                        int32_t G, int64_t N, int64_t K, void* c,
                                        fp8q_out_dtype out, hipStream_t stream);
fp8q_status fp8q_grouped_gemm_rowscaled_precise(const uint8_t* a_q, const float* a_s,
                                                const uint8_t* b_q, const float* b_s, int64_t T,
                                                const int32_t* off, int32_t G, int64_t N,
                                                int64_t K, void* c, fp8q_out_dtype out,
                                                hipStream_t stream);

/*
 * One AdamW step over many tensors, in place.  With g the gradient times
 * *grad_scale (1 where that is NULL) and t the step's number, in FP32:
 *   m = fl(fl(beta1 m) + fl((1 - beta1) g)),
 *   v = fl(fl(beta2 v) + fl((1 - beta2) fl(g g))),
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps);
 * the factors of lr, weight_decay and t are formed in 64 bits and rounded once, and p
 * is within 2^-24 (3 |p| + 8 |update|) of the formula with these m and v.
 *
 * Moments in E4M3 (FP8Q_MOMENTS_E4M3): m holds codes of m and v codes of r = sqrt(v),
 * each 128 consecutive elements of a tensor (the last ones fewer) with one scale,
 * m_s and v_s: fl(amax * fl(1/448)) of their largest finite magnitude amax, multiplier
 * fl(448 * fl(1/amax)) (not finite: scale and codes are 0).  m = code * scale, v =
 * fl(r r), r = code * scale go into the formulas above; then x = fl(m * multiplier)
 * and the same of r are rounded with a dither instead of to the nearest, so that a
 * moment that moves by less than a code's step each time does not stay where it is.
 * |x| becomes the E4M3 value at or below it, or the next one where |x|'s fraction of
 * that step, in units of 2^-20, and u reach 2^20, with
 *   u = (i * 0x85EBCA6B + t * 0x9E3779B1 mod 2^32) >> 12
 * of the element's place i in its tensor and the step's number for m, 2^20 - 1 - u
 * for r; a r that is not zero becomes 2^-9 at least.  (The fraction is of FP32's bits:
 * below 2^-6, of |x| + 2^-6 rounded to FP32.)
 * A m or r that is not finite (of a gradient that is not, or whose square overflows)
 * becomes the code of NaN, 0x7F, with no part in amax: its own parameter is NaN from the
 * next step on at the latest, the others of its group are as without it.
 */
typedef enum {
  FP8Q_MOMENTS_F32 = 0,  /* m, v: float32 [n]                                       */
  FP8Q_MOMENTS_E4M3 = 1  /* m, v: uint8 codes [n]; m_s, v_s: float32 [ceil(n/128)]   */
} fp8q_moments;

typedef struct {
  float* p;       /* master weights [n] (in and out)                                */
  const void* g;  /* gradient [n], float32 or bfloat16                              */
  void* m;        /* first moment (in and out)                                      */
  void* v;        /* second moment, or the codes of its root (in and out)           */
  float* m_s;     /* scales of m and v: E4M3 moments only                           */
  float* v_s;
  void* copy;     /* p as bfloat16 [n] (output), or NULL                            */
  int64_t n;      /* elements, at most 2^34; 0: nothing to do                       */
} fp8q_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;             /* t, 1 for the first step                                */
  const float* lr_dev;      /* DEVICE float32[1] in lr's place, or NULL               */
  const int32_t* step_dev;  /* DEVICE int32[1] (>= 1) in step's place, or NULL        */
  const float* grad_scale;  /* DEVICE float32[1], or NULL                             */
} fp8q_adamw_args;

/*
 *   tensors : HOST array of `count` descriptions, read during the call.
 *   All data pointers 16-byte aligned, scales and the device scalars 4-byte.
 * A captured call keeps host values: a graph that is replayed step after step takes
 * its step's number (and a changing lr) from the device.
 * FP8Q_ERR_UNSUPPORTED: two tensors' p overlap, n > 2^34, a beta outside [0, 1), lr
 * or weight_decay negative or not finite, eps neither 0 nor in [2^-126, 2^125], or
 * step < 1 (without step_dev).
 * No other memory of one call may overlap.
 */
fp8q_status fp8q_adamw(const fp8q_adamw_tensor* tensors, int32_t count,
                       const fp8q_adamw_args* args, fp8q_out_dtype grad_type,
                       fp8q_moments moments, hipStream_t stream);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* fp8q_status_string(fp8q_status status);

/* FP8Q_ABI_VERSION of the loaded library. */
int fp8q_abi_version(void);

/* 1 if the loaded library was built with FP8Q_DEBUG_CHECKS (grouped calls
   synchronize and report invalid device offsets), else 0. */
int fp8q_debug_checks(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_H */
