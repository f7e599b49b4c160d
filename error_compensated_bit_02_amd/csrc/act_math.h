// Device functions that the checkpoint's kernels (activation.hip) and the linear
// layer's (linear.hip) share: the activation functions with their derivatives,
// and eight elements of a checkpoint encoded and decoded.
//
// Activations.  gelu(x) = x*Phi(x) with Phi the normal distribution function;
// gelu_tanh(x) = x*sigma(2u), u = sqrt(2/pi)*(x + 0.044715 x^3), equal to
// 0.5*x*(1 + tanh(u)); silu(x) = x*sigma(x).  With z = |x|/sqrt(2),
// Phi(-|x|) = 0.5*exp(-x^2/2) * P(t), P(t) ~ exp(z^2)*erfc(z), t = 1/(1 + c z), P
// a polynomial of degree 8 without constant term (a least-squares fit with the
// weights moved to the largest errors); the one exponential serves the density
// of the derivative as well.
//
// bf16 (an output step is 2^-8): c = 0.425, P off by at most 1.6e-7 over z in
// [0, 10].  The exponentials' arguments are rounded once, so far out the error
// is theirs: about |a|*2^-24 of exp(a).
// fp32: the arguments' rounding is carried along and multiplied back in, and
// reciprocals get a Newton step.  Within |x| < 1.25 Phi = 0.5 + x*Q(x^2), which
// has no factor to cancel, Q of degree 5 and off by 4.7e-8; beyond, P of degree
// 7 with c = 0.4, off by 3.9e-8 there.  Against 64 bits over [-12, 12], in units
// of 2^-24 of the result, largest measured error: gelu 6.9 below 0 (elementary
// fp32 operations: all of the result) and 2.0 above (2.3), silu 4.5 and 2.6 (2.4
// and 2.0), gelu_tanh 4.4 and 2.7.
#pragma once

#include "activation.h"
#include "internal.h"

#pragma clang fp contract(off)

namespace ob {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

constexpr float kLog2e = 1.4426950408889634f;

// exp(a + low) for a <= 0 in fp32's last bits: the exponential of a's rounded
// base-2 exponent, corrected by what that rounding left out.
__device__ __forceinline__ float exp_fine(float a, float low) {
  constexpr float kLn2 = 0.6931471824645996f, kLn2Low = -1.9046542121259336e-09f;
  const float p = kLog2e * a;
  const float d = __builtin_fmaf(-kLn2Low, p, __builtin_fmaf(-kLn2, p, a)) + low;
  const float e = __builtin_amdgcn_exp2f(p);
  return __builtin_fmaf(e, d, e);
}

// 1/d for finite d >= 1 (of an infinity: 0, but NaN with the Newton step).
template <bool FINE>
__device__ __forceinline__ float reciprocal(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  if constexpr (FINE) return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
  return r;
}

// exp(-|v|).  FINE: 0 from 128 on, and for a NaN, which arrives through the product with x.
template <bool FINE>
__device__ __forceinline__ float exp_falling(float v) {
  if constexpr (FINE) return exp_fine(-fminf(fabsf(v), 128.0f), 0.0f);
  else return __builtin_amdgcn_exp2f(-kLog2e * fabsf(v));
}

// sigma(v) and sigma(v)*(1 - sigma(v)) from e = exp(-|v|), so that neither tail
// cancels or overflows.
template <bool FINE>
__device__ __forceinline__ void sigmoid_slope(float v, float e, float &s, float &ds) {
  const float r = reciprocal<FINE>(1.0f + e);
  const float er = e * r;
  s = v > 0.0f ? r : er;
  ds = er * r;
}

// Phi(x) and exp(-x^2/2).  FINE: past 16 as at 16, where the latter is 0; a NaN as above.
template <bool FINE>
__device__ __forceinline__ void normal_cdf(float x, float &cdf, float &gauss) {
  const float c = FINE ? fminf(fabsf(x), 16.0f) : fabsf(x);
  const float t = reciprocal<FINE>(__builtin_fmaf((FINE ? 0.4f : 0.425f) * 0.70710678118654752f, c, 1.0f));
  if constexpr (FINE) {
    const float half = -0.5f * c, a = c * half;
    gauss = exp_fine(a, __builtin_fmaf(c, half, -a));
    float p = -0.05815780535340309f;     // half of P
    p = __builtin_fmaf(p, t, 0.1218689084053040f);
    p = __builtin_fmaf(p, t, 0.0040680216625332832f);
    p = __builtin_fmaf(p, t, 0.1065559536218643f);
    p = __builtin_fmaf(p, t, 0.0993831828236580f);
    p = __builtin_fmaf(p, t, 0.1133473664522171f);
    p = __builtin_fmaf(p, t, 0.1128134503960610f);
    const float tail = (p * t) * gauss, s = c * c;
    float q = -5.976459760859143e-06f;
    q = __builtin_fmaf(q, s, 0.00010779739386634901f);
    q = __builtin_fmaf(q, s, -0.0011794213205575943f);
    q = __builtin_fmaf(q, s, 0.009969833306968212f);
    q = __builtin_fmaf(q, s, -0.06648973375558853f);
    q = __builtin_fmaf(q, s, 0.3989422619342804f);
    cdf = c < 1.25f ? __builtin_fmaf(x, q, 0.5f) : x > 0.0f ? 1.0f - tail : tail;
  } else {
    gauss = __builtin_amdgcn_exp2f((x * x) * (-0.5f * kLog2e));
    float p = 0.07147843390703201f;
    p = __builtin_fmaf(p, t, -0.3131575882434845f);
    p = __builtin_fmaf(p, t, 0.40761882066726685f);
    p = __builtin_fmaf(p, t, -0.10325203835964203f);
    p = __builtin_fmaf(p, t, 0.25508710741996765f);
    p = __builtin_fmaf(p, t, 0.2007058560848236f);
    p = __builtin_fmaf(p, t, 0.2418406456708908f);
    p = __builtin_fmaf(p, t, 0.23967862129211426f);
    const float tail = 0.5f * (p * t) * gauss;
    cdf = x > 0.0f ? 1.0f - tail : tail;
  }
}

constexpr float kGeluC = 2.0f * 0.79788456080286536f;   // 2 sqrt(2/pi)
constexpr float kGeluK = 0.044715f;

// exp(-|2u|) of gelu_tanh in fp32's last bits: the exponent -|x|*(A + B x^2)
// with what each step's rounding leaves out.  Past 16 as at 16, where it is 0;
// a NaN stays one.
__device__ __forceinline__ float exp_falling_tanh(float x) {
  constexpr float kA = 1.5957691669464111f, kALow = -4.534068054340423e-08f;      // 2 sqrt(2/pi)
  constexpr float kB = 0.07135481387376785f, kBLow = 2.3988324659995897e-09f;     // 0.044715 times that
  const float c = fabsf(x) > 16.0f ? 16.0f : fabsf(x), s = c * c;
  const float b = kB * s, q = kA + b, back = q - kA;
  float low = (kA - (q - back)) + (b - back);      // of the sum
  low += __builtin_fmaf(kB, s, -b);
  low = __builtin_fmaf(kB, __builtin_fmaf(c, c, -s), low);
  low += __builtin_fmaf(kBLow, s, kALow);
  const float a = -c * q;
  return exp_fine(a, __builtin_fmaf(-c, low, __builtin_fmaf(-c, q, -a)));
}

// FINE: for fp32 results.  The plain forms for bf16 are left as they round.
template <int ACT, bool FINE>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == kActGelu) {
    float cdf, gauss;
    normal_cdf<FINE>(x, cdf, gauss);
    return x * cdf;
  } else if constexpr (FINE) {
    float s, ds;
    sigmoid_slope<true>(x, ACT == kActGeluTanh ? exp_falling_tanh(x) : exp_falling<true>(x), s, ds);
    return x * s;
  } else {
    const float v = ACT == kActGeluTanh ? kGeluC * x * __builtin_fmaf(kGeluK * x, x, 1.0f) : x;
    return x * reciprocal<false>(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v));
  }
}

// The derivative.  Where the factor beside sigma*(1 - sigma) could overflow
// while that product is 0, it is bounded (a NaN of x arrives through sigma).
template <int ACT, bool FINE>
__device__ __forceinline__ float act_slope(float x) {
  float s, ds;
  if constexpr (ACT == kActGelu) {
    normal_cdf<FINE>(x, s, ds);
    return __builtin_fmaf(x * 0.39894228040143268f, ds, s);
  } else if constexpr (ACT == kActGeluTanh) {
    const float v = kGeluC * x * __builtin_fmaf(kGeluK * x, x, 1.0f);
    sigmoid_slope<FINE>(v, FINE ? exp_falling_tanh(x) : exp_falling<false>(v), s, ds);
    const float c = __builtin_amdgcn_fmed3f(x, -64.0f, 64.0f);
    return __builtin_fmaf(ds, kGeluC * c * __builtin_fmaf(3.0f * kGeluK * c, c, 1.0f), s);
  } else {
    sigmoid_slope<FINE>(x, exp_falling<FINE>(x), s, ds);
    return __builtin_fmaf(ds, x, s);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  bf16x2 r;
  r[0] = static_cast<__bf16>(a);
  r[1] = static_cast<__bf16>(b);
  return __builtin_bit_cast(uint32_t, r);
}

// The factor that encode8 takes for a scale byte.  A block that is not finite:
// NaN * x encodes as the NaN code of e4m3; int8 codes are 0 there.
template <int FMT>
__device__ __forceinline__ float act_inverse(uint32_t s) {
  return s == kNanScale ? (FMT == kE4M3 ? __uint_as_float(0x7fc00000u) : 0.0f) : __uint_as_float((254u - s) << 23);
}

// The codes of eight elements, to nearest even.
template <int FMT>
__device__ __forceinline__ u32x2 encode8(const float (&v)[8], const float (&inv)[8]) {
  u32x2 w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = __builtin_amdgcn_fmed3f(v[4 * h + k], -__uint_as_float(kTopBits), __uint_as_float(kTopBits));
    if constexpr (FMT == kE4M3) {
      int c = __builtin_amdgcn_cvt_pk_fp8_f32(q[0] * inv[4 * h], q[1] * inv[4 * h + 1], 0, false);
      c = __builtin_amdgcn_cvt_pk_fp8_f32(q[2] * inv[4 * h + 2], q[3] * inv[4 * h + 3], c, true);
      w[h] = static_cast<uint32_t>(c);
    } else {
      uint32_t c = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        c |= (static_cast<uint32_t>(static_cast<int>(rintf(q[k] * inv[4 * h + k]))) & 0xffu) << (8 * k);
      w[h] = c;
    }
  }
  return w;
}

// The fp32 scale of a scale byte, NaN for a block that is not finite.
__device__ __forceinline__ float act_scale_or_nan(uint32_t b) {
  return b == kNanScale ? __uint_as_float(0x7fc00000u) : act_scale_value(b);
}

template <int FMT>
__device__ __forceinline__ void decode8(u32x2 w, const float (&s)[8], float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = w[h];
    if constexpr (FMT == kE4M3) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
      x[4 * h] = lo[0] * s[4 * h];
      x[4 * h + 1] = lo[1] * s[4 * h + 1];
      x[4 * h + 2] = hi[0] * s[4 * h + 2];
      x[4 * h + 3] = hi[1] * s[4 * h + 3];
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[4 * h + k] = static_cast<float>(static_cast<int>(__builtin_amdgcn_sbfe(c, 8 * k, 8))) * s[4 * h + k];
    }
  }
}

}  // namespace ob
