// 8-bit activation checkpoints (gfx950): save (with the activation in the
// same pass), load, and the activation's backward from the checkpoint.  The
// format and its reasons are in activation.h.
//
// All three are bound by HBM: gelu's backward of 16384 x 8192 in bf16 moves 675
// MB in 128 us (5.3 TB/s, a plain copy's rate), with the 30-odd vector
// instructions an element of its derivative close behind (fp32: 4.8 TB/s).  A tile is one scale
// block (32 rows) of 128 columns: a lane owns 8 columns 8*(l%16) of every fourth
// row, so every row access is a full 16-byte vector per lane, a block's scales
// are read or formed once for the lane's rows, and the largest magnitude of a
// column needs two lane exchanges.
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
#include "internal.h"
#include "activation.h"

#pragma clang fp contract(off)

namespace ob {
namespace {

constexpr int kCols = 128;          // columns of a tile
// A tile is a wavefront's, eight rows a lane; where fp32 activations are
// computed, with half as many instructions again as bf16's, it is a workgroup's,
// two rows a lane.  gelu and save, fp32, 333 x 1000: 5.1 us against 10.5 a
// wavefront a tile (7.1 with the bf16 forms), 4096 x 4096 33 against 42, 16384 x
// 8192 217 against 232; its backward 4.3 against 9.7, 32 against 39, 220 against 224.
template <typename T, int ACT>
constexpr bool kSplit = sizeof(T) == 4 && ACT != kActNone;
template <bool SPLIT>
constexpr int kRowsPerLane = SPLIT ? kActBlock / 4 / kWaves : kActBlock / 4;
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

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  bf16x2 r;
  r[0] = static_cast<__bf16>(a);
  r[1] = static_cast<__bf16>(b);
  return __builtin_bit_cast(uint32_t, r);
}

// Eight consecutive elements as fp32: 16-byte accesses where the row allows
// them and all eight exist, single elements otherwise (absent ones read as 0).
// Everything is streamed once, so the accesses are non-temporal: 5-12% faster
// at 16384 x 8192 in bf16 (save and load with gelu_tanh 210 -> 184 us, gelu_tanh's
// backward 146 -> 136 us; most of it from the stores).
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, int n, float (&v)[8]) {
  if (VEC && n >= 8) {
    constexpr int kEach = 16 / sizeof(T);
#pragma unroll
    for (int k = 0; k < 8; k += kEach) {
      const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + k));
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if constexpr (sizeof(T) == 4) {
          v[k + h] = __uint_as_float(w[h]);
        } else {
          v[k + 2 * h] = __uint_as_float(w[h] << 16);
          v[k + 2 * h + 1] = __uint_as_float(w[h] & 0xffff0000u);
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = 0.0f;
      if (k < n) {
        if constexpr (sizeof(T) == 4) v[k] = p[k];
        else v[k] = __uint_as_float(static_cast<uint32_t>(p[k]) << 16);
      }
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, int n, const float (&v)[8]) {
  if (VEC && n >= 8) {
    constexpr int kEach = 16 / sizeof(T);
#pragma unroll
    for (int k = 0; k < 8; k += kEach) {
      u32x4 w;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if constexpr (sizeof(T) == 4) w[h] = __float_as_uint(v[k + h]);
        else w[h] = pack_bf16(v[k + 2 * h], v[k + 2 * h + 1]);
      }
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(p + k));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k < n) {
        if constexpr (sizeof(T) == 4) p[k] = v[k];
        else p[k] = static_cast<uint16_t>(pack_bf16(v[k], 0.0f));
      }
    }
  }
}

// This lane's part of its tile: first row (the others follow at steps of four),
// first column, number of columns; false where nothing is left to do.
struct Place {
  int64_t row;
  int col;
  int n;
  int64_t block;
};

template <bool SPLIT>
__device__ __forceinline__ bool place(const ActArgs &a, Place &at) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = SPLIT ? blockIdx.y * gridDim.x + blockIdx.x : blockIdx.x * kWaves + wave;
  if (tile >= a.tiles) return false;
  const uint32_t blk = tile / a.col_tiles, ct = tile - blk * a.col_tiles;
  const int lane = threadIdx.x & 63;
  at.block = blk;
  at.row = static_cast<int64_t>(blk) * kActBlock + (lane >> 4) + (SPLIT ? wave * 4 * kRowsPerLane<true> : 0);
  at.col = static_cast<int>(ct) * kCols + (lane & 15) * 8;
  at.n = static_cast<int>(a.cols - at.col);
  return true;
}

template <typename T, int FMT, int ACT, bool VEC>
__global__ __launch_bounds__(kBlock) void act_save_kernel(const ActArgs a) {
  Place at;
  constexpr bool SPLIT = kSplit<T, ACT>;
  constexpr int kRows = kRowsPerLane<SPLIT>;
  if (!place<SPLIT>(a, at)) return;
  float v[kRows][8];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t r = at.row + 4 * j;
    load8<T, VEC>(static_cast<const T *>(a.x) + r * a.ldx + at.col, r < a.rows ? at.n : 0, v[j]);
  }
  uint32_t top[8], scale[8];
  float inv[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kRows; ++j) m = max(m, __float_as_uint(v[j][k]) & 0x7fffffffu);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
    top[k] = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
  }
  if constexpr (SPLIT) {     // the largest of the workgroup's wavefronts
    __shared__ uint32_t tops[kWaves][kCols];
    const int c = (threadIdx.x & 15) * 8;
    if ((threadIdx.x & 48) == 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) tops[threadIdx.x >> 6][c + k] = top[k];
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
#pragma unroll
      for (int k = 0; k < 8; ++k) top[k] = max(top[k], tops[w][c + k]);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    scale[k] = act_scale<FMT>(top[k]);
    // a NaN block: NaN * x encodes as the NaN code of e4m3; int8 codes are 0 there
    inv[k] = scale[k] == kNanScale ? (FMT == kE4M3 ? __uint_as_float(0x7fc00000u) : 0.0f)
                                   : __uint_as_float((254u - scale[k]) << 23);
  }
  if (at.n <= 0) return;
  uint8_t *codes = a.codes + at.col;
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t r = at.row + 4 * j;
    if (r >= a.rows) break;
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        q[k] = __builtin_amdgcn_fmed3f(v[j][4 * h + k], -__uint_as_float(kTopBits), __uint_as_float(kTopBits));
      }
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
    uint8_t *out = codes + r * a.pitch;
    if (at.n >= 8) {
      *reinterpret_cast<uint2 *>(out) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (k < at.n) out[k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
    }
    if constexpr (ACT != kActNone) {
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = act_value<ACT, sizeof(T) == 4>(v[j][k]);
      store8<T, VEC>(static_cast<T *>(a.y) + r * a.ldy + at.col, at.n, y);
    }
  }
  if ((threadIdx.x & (SPLIT ? ~15u : 48u)) == 0) {
    uint8_t *out = a.scales + at.block * a.pitch + at.col;
    if (at.n >= 8) {
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k >> 2] |= scale[k] << (8 * (k & 3));
      *reinterpret_cast<uint2 *>(out) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (k < at.n) out[k] = static_cast<uint8_t>(scale[k]);
    }
  }
}

// The lane's eight scales: reading whole groups of eight is in bounds, the
// pitch being a multiple of 64.
template <int FMT>
__device__ __forceinline__ void load_scales(const ActArgs &a, const Place &at, float (&s)[8]) {
  const uint2 w = *reinterpret_cast<const uint2 *>(a.scales_in + at.block * a.pitch + at.col);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t b = ((k < 4 ? w.x : w.y) >> (8 * (k & 3))) & 0xffu;
    s[k] = b == kNanScale ? __uint_as_float(0x7fc00000u) : act_scale_value(b);
  }
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

// ACT == kActNone: out = the checkpoint's values; otherwise out = dy * act'(values).
template <typename T, int FMT, int ACT, bool VEC>
__global__ __launch_bounds__(kBlock) void act_read_kernel(const ActArgs a) {
  Place at;
  constexpr bool SPLIT = kSplit<T, ACT>;
  constexpr int kRows = kRowsPerLane<SPLIT>;
  if (!place<SPLIT>(a, at) || at.n <= 0) return;
  float s[8];
  load_scales<FMT>(a, at, s);
  u32x2 w[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t r = at.row + 4 * j;
    w[j] = u32x2{0, 0};
    if (r < a.rows) w[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(a.codes_in + r * a.pitch + at.col));
  }
  float g[kRows][8];
  if constexpr (ACT != kActNone) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int64_t r = at.row + 4 * j;
      load8<T, VEC>(static_cast<const T *>(a.x) + r * a.ldx + at.col, r < a.rows ? at.n : 0, g[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t r = at.row + 4 * j;
    if (r >= a.rows) break;
    __builtin_amdgcn_sched_barrier(0);    // a row at a time: decoding all rows first takes registers for nothing
    float x[8];
    decode8<FMT>(w[j], s, x);
    if constexpr (ACT != kActNone) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = g[j][k] * act_slope<ACT, sizeof(T) == 4>(x[k]);
    }
    store8<T, VEC>(static_cast<T *>(a.y) + r * a.ldy + at.col, at.n, x);
  }
}

// Vector accesses need every row to start on 16 bytes.
bool vector_rows(const ActArgs &a, int size) {
  return (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y)) % 16 == 0 &&
         (a.ldx * size) % 16 == 0 && (a.ldy * size) % 16 == 0;
}

template <typename T, int FMT, int ACT>
void by_rows(bool save, const ActArgs &a, hipStream_t s) {
  // up to kWaves * kMaxGrid tiles
  const uint32_t ny = kSplit<T, ACT> ? static_cast<uint32_t>((a.tiles + kMaxGrid - 1) / kMaxGrid) : kWaves;
  const dim3 grid((a.tiles + ny - 1) / ny, kSplit<T, ACT> ? ny : 1);
  const bool vec = vector_rows(a, sizeof(T));
  if (save) {
    if (vec) act_save_kernel<T, FMT, ACT, true><<<grid, kBlock, 0, s>>>(a);
    else act_save_kernel<T, FMT, ACT, false><<<grid, kBlock, 0, s>>>(a);
  } else {
    if (vec) act_read_kernel<T, FMT, ACT, true><<<grid, kBlock, 0, s>>>(a);
    else act_read_kernel<T, FMT, ACT, false><<<grid, kBlock, 0, s>>>(a);
  }
}

template <typename T, int FMT>
void by_act(bool save, int act, const ActArgs &a, hipStream_t s) {
  if (act == kActGelu) by_rows<T, FMT, kActGelu>(save, a, s);
  else if (act == kActGeluTanh) by_rows<T, FMT, kActGeluTanh>(save, a, s);
  else if (act == kActSilu) by_rows<T, FMT, kActSilu>(save, a, s);
  else by_rows<T, FMT, kActNone>(save, a, s);
}

}  // namespace

int64_t act_tiles(int64_t rows, int64_t cols) {
  return act_blocks(rows) * ((cols + kCols - 1) / kCols);
}

void launch_act(bool save, int fmt, int act, bool bf16, ActArgs a, hipStream_t s) {
  a.col_tiles = static_cast<uint32_t>((a.cols + kCols - 1) / kCols);
  a.tiles = static_cast<uint32_t>(act_tiles(a.rows, a.cols));
  a.pitch = act_pitch(a.cols);
  if (bf16) {
    if (fmt == kE4M3) by_act<uint16_t, kE4M3>(save, act, a, s);
    else by_act<uint16_t, kInt8>(save, act, a, s);
  } else {
    if (fmt == kE4M3) by_act<float, kE4M3>(save, act, a, s);
    else by_act<float, kInt8>(save, act, a, s);
  }
}

}  // namespace ob
