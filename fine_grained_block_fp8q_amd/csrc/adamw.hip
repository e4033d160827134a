// One AdamW step over many tensors.
//
// Per element, with t the step's number and g the gradient (times grad_scale):
//   m' = fl(fl(b1 m) + fl((1 - b1) g)),  v' = fl(fl(b2 v) + fl((1 - b2) fl(g g))),
//   p' = p (1 - lr wd) - lr/(1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps),
// masters in FP32, moments in FP32 or in 8 bits.  Bound by memory: a master is
// read and written (8 bytes), the gradient read (2 or 4), the moments read and
// written (16, or 4 and the scales), the BF16 copy written (2).  44M parameters,
// moments in FP32, BF16 gradients and copy: 195 to 199 us (6.2 TB/s); 340M, moments in
// 8 bits: 921 to 932 us (5.9 TB/s), near which the vector ALU's work comes too.
//
// Moments in 8 bits: E4M3 codes of m' and of sqrt(v') (the root has half the
// exponent range of v', so 128 elements of one scale reach 2^35 down from the
// largest v'), 128 consecutive elements a scale: amax fl(1/448), the codes those of
// the values times 448 fl(1/amax) (one division a group).  The codes are not rounded
// to the nearest: a moment moves by a small part of itself a step (5% of v' at b2 =
// 0.95, 2.5% of its root), less than half of E4M3's step, and would never leave its
// code.  Each magnitude x is rounded up where its fraction of a step and a dither u
// reach 1, u = frac(t phi + i psi) in 20 bits with i the element's place in its
// tensor: over the steps of one element the u are spread evenly, so that the codes of
// a value that stands have its mean.  (A moment feeds back into the next step, whose u
// is related: under a constant gradient the codes' mean is off by 0.3% on average and
// 1.4% at most, against 0 and 1.6% of independent u.)  A root that is not zero keeps a
// code that is not zero: m' is never divided by eps alone.  A moment that is not finite
// has no place in amax: it would take its group's 127 others with it.
//
// A workgroup of 256 lanes takes 2048 consecutive elements of one tensor, 16 lanes
// (a DPP row) a group.  Up to 64 tensors (56 with their scales) go out in one launch,
// described in its arguments; a workgroup finds its tensor from the tensors' first
// workgroups, one a lane.  The host writes arguments slowly (a launch alone takes 6 us
// more for each KiB of them, and 20 more past 4 KiB), so there are launches of 8, 24
// and 64 (60 tensors of 4096 elements: 6.6 us one after the other, 18.4 alone).

#include <math.h>

#include <type_traits>

#include "activation.hpp"
#include "fp8q.h"
#include "launch.hpp"
#include "fp8q_device.hpp"

namespace fp8q {

constexpr int kThreads = 256;
constexpr int kElems = 2048;   // of one workgroup
static_assert((int64_t(1) << 34) / kElems <= max_blocks(kThreads), "the largest tensor in a launch");

struct Moments32 {
  float* p;
  const void* g;
  void* m;
  void* v;
  void* copy;
  int64_t n;
};
struct Moments8 : Moments32 {
  float* m_s;
  float* v_s;
};
template <bool E4M3>
using Tensor = typename std::conditional<E4M3, Moments8, Moments32>::type;

struct AdamwScalars {
  const float* lr;  // on the device, or NULL
  const int32_t* step;
  const float* grad_scale;
  double log_b1, log_b2, lr_host, decay, c1;  // c1: 1 - b1^t
  float b1, one_b1, b2, one_b2, eps;
  float keep, rate, inv_root;  // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t dither;             // t's part of the dither
};

template <bool E4M3, int CAP>
struct AdamwLaunch {
  AdamwScalars s;
  int32_t first[CAP];  // first workgroup of each tensor; past the last, INT32_MAX
  Tensor<E4M3> t[CAP];
};

constexpr uint32_t kDitherStep = 0x9E3779B1u, kDitherPlace = 0x85EBCA6Bu;

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// |x| <= 448 (1 + 2^-23) rounded to E4M3 with the dither's 20 bits u: the step of
// E4M3 is the 20th bit of an FP32 value; below 2^-6, of the value 2^-6 higher.
__device__ __forceinline__ float dithered(float x, uint32_t u) {
  const float up = x < 0x1p-6f ? 0x1p-6f : 0.f;
  return fminf(__uint_as_float((__float_as_uint(x + up) + u) & ~0xFFFFFu) - up, kE4M3Max);
}

// The correctly rounded root of x, 0 or at least 2^-96 (below, the products here could
// lose bits): of the instruction's value, an ulp off at most, and its neighbours the
// one whose square is nearest.
__device__ __forceinline__ float root_of_normal(float x) {
  float s = __builtin_amdgcn_sqrtf(x);
  const float lo = __uint_as_float(__float_as_uint(s) - 1);
  const float hi = __uint_as_float(__float_as_uint(s) + 1);
  const float below = __builtin_fmaf(-lo, s, x), above = __builtin_fmaf(-hi, s, x);
  s = below <= 0.f ? lo : s;
  return above > 0.f ? hi : s;
}

// Scale and multiplier of a group of moments, 0 where the multiplier is not finite.
struct MomentRule {
  float mul, s;
};
__device__ __forceinline__ MomentRule moment_rule(float amax) {
  const float mul = kE4M3Max * (1.f / amax);
  const bool flushed = !__builtin_isfinite(mul);
  return {flushed ? 0.f : mul, flushed ? 0.f : amax * (1.f / kE4M3Max)};
}

// max(m, |a|, |b|), a NaN where one of them is.
__device__ __forceinline__ float maximum3abs(float m, float a, float b) {
  float r;
  asm("v_maximum3_f32 %0, %1, |%2|, |%3|" : "=v"(r) : "v"(m), "v"(a), "v"(b));
  return r;
}

// A lane's eight elements, in two fours.
struct Eight {
  v4f v[2];
};

__device__ __forceinline__ v4f unpack_e4m3x4(uint32_t w) {
  return v4f{__builtin_amdgcn_cvt_f32_fp8((int)w, 0), __builtin_amdgcn_cvt_f32_fp8((int)w, 1),
             __builtin_amdgcn_cvt_f32_fp8((int)w, 2), __builtin_amdgcn_cvt_f32_fp8((int)w, 3)};
}

__device__ __forceinline__ v4f unpack_bf16x4(uint32_t lo, uint32_t hi) {
  return v4f{bf16_lo(lo), bf16_hi(lo), bf16_lo(hi), bf16_hi(hi)};
}

__device__ __forceinline__ v2u pack_bf16x4(const v4f& v) {
  return v2u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

template <bool E4M3_MOMENTS, bool BF16_GRAD, int CAP>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamwLaunch<E4M3_MOMENTS, CAP> l) {
  const AdamwScalars& a = l.s;
  const int lane = threadIdx.x & 63;
  const int bid = (int)blockIdx.x;
  const uint64_t upto = __ballot(lane < CAP && l.first[lane < CAP ? lane : 0] <= bid);
  const int ti = __builtin_amdgcn_readfirstlane(__builtin_popcountll(upto) - 1);
  const Tensor<E4M3_MOMENTS> t = l.t[ti];
  const int64_t base = (int64_t)(bid - l.first[ti]) * kElems;
  const int rest = t.n - base < kElems ? (int)(t.n - base) : kElems;  // of the workgroup
  // (uniform bases, offsets of 32 bits)
  float* const tp = t.p + base;
  const float* const g32 = static_cast<const float*>(t.g) + base;
  const uint16_t* const g16 = static_cast<const uint16_t*>(t.g) + base;
  float *const m32 = static_cast<float*>(t.m) + base, *const v32 = static_cast<float*>(t.v) + base;
  uint8_t *const m8 = static_cast<uint8_t*>(t.m) + base, *const v8 = static_cast<uint8_t*>(t.v) + base;
  uint16_t* const copy = t.copy ? static_cast<uint16_t*>(t.copy) + base : nullptr;

  float keep = a.keep, rate = a.rate, inv_root = a.inv_root;
  uint32_t step_dither = a.dither;
  if (a.step || a.lr) {
    const double lr = a.lr ? (double)*a.lr : a.lr_host;
    keep = (float)(1.0 - lr * a.decay);
    if (a.step) {
      const int32_t st = *a.step;
      rate = (float)(lr / -expm1((double)st * a.log_b1));
      inv_root = (float)(1.0 / sqrt(-expm1((double)st * a.log_b2)));
      step_dither = (uint32_t)st * kDitherStep;
    } else {
      rate = (float)(lr / a.c1);
    }
  }
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;

  // The lane's two fours lie 64 apart, so that 16 lanes' accesses of FP32 are 256
  // consecutive bytes (340M parameters with moments in 8 bits: 935 us, with eight
  // consecutive elements a lane 1010).
  const uint32_t l16 = lane & 15, group = (threadIdx.x >> 4) * kGroup;
  if ((int)group >= rest) return;  // (whole DPP rows)
  constexpr uint32_t kApart = 64;
  const uint32_t o = group + 4 * l16;
  const bool whole = (int)group + kGroup <= rest;
  auto at = [&](int h, int j) { return o + kApart * h + j; };
  auto live = [&](int h, int j) { return (int)at(h, j) < rest; };
  // Streams of 16 bytes a lane, and what is only written, pass the caches by (one layer,
  // moments in FP32: 197 us; with the gradients' 8 bytes too 204, with none 229).
  Eight p, g, m, v;
  if (whole) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      p.v[h] = __builtin_nontemporal_load(reinterpret_cast<const v4f*>(tp + at(h, 0)));
    if constexpr (!BF16_GRAD) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        g.v[h] = __builtin_nontemporal_load(reinterpret_cast<const v4f*>(g32 + at(h, 0)));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v2u w = *reinterpret_cast<const v2u*>(g16 + at(h, 0));
        g.v[h] = unpack_bf16x4(w[0], w[1]);
      }
    }
    if constexpr (E4M3_MOMENTS) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m.v[h] = unpack_e4m3x4(*reinterpret_cast<const uint32_t*>(m8 + at(h, 0)));
        v.v[h] = unpack_e4m3x4(*reinterpret_cast<const uint32_t*>(v8 + at(h, 0)));
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m.v[h] = __builtin_nontemporal_load(reinterpret_cast<const v4f*>(m32 + at(h, 0)));
        v.v[h] = __builtin_nontemporal_load(reinterpret_cast<const v4f*>(v32 + at(h, 0)));
      }
    }
  } else {  // the tensor's last group: element by element, zeros past its end
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t i = at(h, j);
        const bool in = live(h, j);
        p.v[h][j] = in ? tp[i] : 0.f;
        g.v[h][j] = !in ? 0.f : BF16_GRAD ? __uint_as_float((uint32_t)g16[i] << 16) : g32[i];
        if constexpr (E4M3_MOMENTS) {
          m.v[h][j] = in ? __builtin_amdgcn_cvt_f32_fp8((int)m8[i], 0) : 0.f;
          v.v[h][j] = in ? __builtin_amdgcn_cvt_f32_fp8((int)v8[i], 0) : 0.f;
        } else {
          m.v[h][j] = in ? m32[i] : 0.f;
          v.v[h][j] = in ? v32[i] : 0.f;
        }
      }
  }
  const int64_t gi = base / kGroup + (threadIdx.x >> 4);
  float ms = 1.f, vs = 1.f;
  if constexpr (E4M3_MOMENTS) {
    ms = t.m_s[gi];
    vs = t.v_s[gi];
  }

  Eight root;
  bool small = false;  // some v is below what root_of_normal() takes
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = g.v[h][j] * gs;
      float m0 = m.v[h][j], v0 = v.v[h][j];
      if constexpr (E4M3_MOMENTS) {
        m0 = m0 * ms;
        const float r = v0 * vs;
        v0 = r * r;
      }
      m.v[h][j] = m0 * a.b1 + x * a.one_b1;
      const float vn = v0 * a.b2 + (x * x) * a.one_b2;
      v.v[h][j] = vn;
      small = small || (vn < 0x1p-96f && vn != 0.f);
    }
  if (__ballot(small) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) root.v[h][j] = root_of_normal(v.v[h][j]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) root.v[h][j] = __builtin_sqrtf(v.v[h][j]);
  }
  // (The update's quotient by the reciprocal instruction, an ulp off at most.)
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float den = __builtin_fmaf(root.v[h][j], inv_root, a.eps);
      const float quotient = m.v[h][j] * __builtin_amdgcn_rcpf(den);
      p.v[h][j] = __builtin_fmaf(-rate, quotient, p.v[h][j] * keep);
    }

  uint32_t mq[2], vq[2];
  if constexpr (E4M3_MOMENTS) {
    float am = 0.f, av = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        am = maximum3abs(am, m.v[h][j], m.v[h][j + 1]);
        av = maximum3abs(av, root.v[h][j], root.v[h][j + 1]);
      }
    // Moments that are not finite: rare, the wave looks for them one by one.
    const bool lost = __ballot(!__builtin_isfinite(am) || !__builtin_isfinite(av)) != 0;
    if (lost) {
      am = av = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (__builtin_isfinite(m.v[h][j])) am = fmaxf(am, fabsf(m.v[h][j]));
          if (__builtin_isfinite(root.v[h][j])) av = fmaxf(av, root.v[h][j]);
        }
    }
    const MomentRule rm = moment_rule(row16_max(am)), rv = moment_rule(row16_max(av));
    const uint32_t place = ((uint32_t)base + o) * kDitherPlace + step_dither;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4f cm, cv;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = (place + (kApart * h + j) * kDitherPlace) >> 12;
        const float x = m.v[h][j] * rm.mul, y = root.v[h][j] * rv.mul;
        cm[j] = copysignf(dithered(fabsf(x), u), x);
        const float d = dithered(y, 0xFFFFFu - u);
        cv[j] = d == 0.f && y > 0.f ? 0x1p-9f : d;
      }
      mq[h] = pack_e4m3x4(cm[0], cm[1], cm[2], cm[3]);
      vq[h] = pack_e4m3x4(cv[0], cv[1], cv[2], cv[3]);
    }
    if (lost) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t byte = 0xFFu << (8 * j), nan = 0x7Fu << (8 * j);
          if (!__builtin_isfinite(m.v[h][j])) mq[h] = (mq[h] & ~byte) | nan;
          if (!__builtin_isfinite(root.v[h][j])) vq[h] = (vq[h] & ~byte) | nan;
        }
    }
    if (l16 == 0) {
      t.m_s[gi] = rm.s;
      t.v_s[gi] = rv.s;
    }
  }

  if (whole) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      __builtin_nontemporal_store(p.v[h], reinterpret_cast<v4f*>(tp + at(h, 0)));
    if constexpr (E4M3_MOMENTS) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<uint32_t*>(m8 + at(h, 0)) = mq[h];
        *reinterpret_cast<uint32_t*>(v8 + at(h, 0)) = vq[h];
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __builtin_nontemporal_store(m.v[h], reinterpret_cast<v4f*>(m32 + at(h, 0)));
        __builtin_nontemporal_store(v.v[h], reinterpret_cast<v4f*>(v32 + at(h, 0)));
      }
    }
    if (copy) {
      const v2u lo = pack_bf16x4(p.v[0]), hi = pack_bf16x4(p.v[1]);
      __builtin_nontemporal_store(lo, reinterpret_cast<v2u*>(copy + at(0, 0)));
      __builtin_nontemporal_store(hi, reinterpret_cast<v2u*>(copy + at(1, 0)));
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!live(h, j)) continue;
        const uint32_t i = at(h, j);
        tp[i] = p.v[h][j];
        if constexpr (E4M3_MOMENTS) {
          m8[i] = (uint8_t)(mq[h] >> (8 * j));
          v8[i] = (uint8_t)(vq[h] >> (8 * j));
        } else {
          m32[i] = m.v[h][j];
          v32[i] = v.v[h][j];
        }
        if (copy) copy[i] = (uint16_t)pack_bf16x2(p.v[h][j], 0.f);
      }
  }
}

// Tensors tensors[i], tensors[i + 1], ... in one launch, as many as fit; i becomes the
// first that did not.
template <bool E4M3, bool BF16_GRAD, int CAP>
static hipError_t launch(const AdamwScalars& s, const fp8q_adamw_tensor* tensors, int32_t count,
                         int32_t& i, hipStream_t stream) {
  AdamwLaunch<E4M3, CAP> a;
  a.s = s;
  int k = 0;
  int64_t blocks = 0;
  for (; i < count && k < CAP; ++i) {
    const fp8q_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const int64_t b = (t.n + kElems - 1) / kElems;
    if (blocks + b > max_blocks(kThreads)) break;
    Tensor<E4M3>& to = a.t[k];
    to.p = t.p;
    to.g = t.g;
    to.m = t.m;
    to.v = t.v;
    to.copy = t.copy;
    to.n = t.n;
    if constexpr (E4M3) {
      to.m_s = t.m_s;
      to.v_s = t.v_s;
    }
    a.first[k++] = (int32_t)blocks;
    blocks += b;
  }
  if (k == 0) return hipSuccess;
  for (int j = k; j < CAP; ++j) {
    a.first[j] = 0x7FFFFFFF;
    a.t[j] = Tensor<E4M3>{};
  }
  hipLaunchKernelGGL((adamw_kernel<E4M3, BF16_GRAD, CAP>), dim3((unsigned)blocks), dim3(kThreads),
                     0, stream, a);
  return hipGetLastError();
}

template <bool E4M3, bool BF16_GRAD>
static hipError_t launches(const AdamwScalars& s, const fp8q_adamw_tensor* tensors, int32_t count,
                           hipStream_t stream) {
  constexpr int kMost = E4M3 ? 56 : 64;  // of 4 KiB of arguments
  static_assert(sizeof(AdamwLaunch<E4M3, kMost>) <= 4096, "the arguments of a launch");
  int32_t i = 0;
  hipError_t e = hipSuccess;
  while (i < count && e == hipSuccess) {
    const int32_t left = count - i;
    e = left <= 8    ? launch<E4M3, BF16_GRAD, 8>(s, tensors, count, i, stream)
        : left <= 24 ? launch<E4M3, BF16_GRAD, 24>(s, tensors, count, i, stream)
                     : launch<E4M3, BF16_GRAD, kMost>(s, tensors, count, i, stream);
  }
  return e;
}

hipError_t launch_adamw(const fp8q_adamw_tensor* tensors, int32_t count, const fp8q_adamw_args& h,
                        int grad_bf16, int e4m3, hipStream_t stream) {
  AdamwScalars a;
  a.lr = h.lr_dev;
  a.step = h.step_dev;
  a.grad_scale = h.grad_scale;
  a.log_b1 = log(h.beta1);
  a.log_b2 = log(h.beta2);
  a.lr_host = h.lr;
  a.decay = h.weight_decay;
  a.b1 = (float)h.beta1;
  a.one_b1 = (float)(1.0 - h.beta1);
  a.b2 = (float)h.beta2;
  a.one_b2 = (float)(1.0 - h.beta2);
  a.eps = (float)h.eps;
  a.keep = (float)(1.0 - h.lr * h.weight_decay);
  // 1 - beta^t cancels for a beta near 1: from the logarithm, in 64 bits
  const double c2 = -expm1((double)h.step * a.log_b2);
  a.c1 = -expm1((double)h.step * a.log_b1);
  a.rate = (float)(h.lr / a.c1);
  a.inv_root = (float)(1.0 / sqrt(c2));
  a.dither = (uint32_t)h.step * kDitherStep;
  auto f = e4m3 ? (grad_bf16 ? launches<true, true> : launches<true, false>)
                : (grad_bf16 ? launches<false, true> : launches<false, false>);
  return f(a, tensors, count, stream);
}

}  // namespace fp8q
