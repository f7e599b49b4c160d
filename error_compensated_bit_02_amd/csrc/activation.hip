// 8-bit activation checkpoints (gfx950): save (with the activation in the
// same pass), load, and the activation's backward from the checkpoint.  The
// format and its reasons are in activation.h.
//
// All three are bound by HBM: gelu's backward of 16384 x 8192 in bf16 moves 675
// MB in 136 us (5.0 TB/s, a plain copy's rate), with the 30-odd vector
// instructions an element of its derivative close behind.  One wavefront handles one scale block (32 rows)
// of 128 columns: lane l owns the 8 columns 8*(l%16) of rows l/16 + 4*j,
// j < 8, so every row access is a full 16-byte vector per lane, a block's
// scales are read or formed once per 8 rows, and the largest magnitude of a
// column needs two lane exchanges.
//
// Activations.  gelu(x) = x*Phi(x) with Phi the normal distribution function;
// gelu_tanh(x) = x*sigma(2u), u = sqrt(2/pi)*(x + 0.044715 x^3), equal to
// 0.5*x*(1 + tanh(u)); silu(x) = x*sigma(x).  With z = |x|/sqrt(2),
// Phi(-|x|) = 0.5*exp(-x^2/2) * P(t), P(t) ~ exp(z^2)*erfc(z), t = 1/(1 + 0.425 z):
// P is a degree-8 polynomial without constant term fitted to relative error
// 1.5e-7 over z in [0, 10] (a least-squares fit with the weights moved to the
// largest errors), so the tail keeps its relative accuracy, and the one
// exponential serves the density of the derivative as well.
#include "internal.h"
#include "activation.h"

#pragma clang fp contract(off)

namespace ob {
namespace {

constexpr int kCols = 128;          // columns of a wavefront's tile
constexpr int kRowsPerLane = 8;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v));
}

// sigma(v) and sigma(v)*(1 - sigma(v)), the latter from exp(-|v|) so that
// neither tail cancels or overflows.
__device__ __forceinline__ void sigmoid_slope(float v, float &s, float &ds) {
  const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(v));
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  const float er = e * r;
  s = v > 0.0f ? r : er;
  ds = er * r;
}

// Phi(x) and exp(-x^2/2).
__device__ __forceinline__ void normal_cdf(float x, float &cdf, float &gauss) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.425f * 0.70710678118654752f, fabsf(x), 1.0f));
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

constexpr float kGeluC = 2.0f * 0.79788456080286536f;   // 2 sqrt(2/pi)
constexpr float kGeluK = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == kActGelu) {
    float cdf, gauss;
    normal_cdf(x, cdf, gauss);
    return x * cdf;
  } else if constexpr (ACT == kActGeluTanh) {
    return x * sigmoid(kGeluC * x * __builtin_fmaf(kGeluK * x, x, 1.0f));
  } else {
    return x * sigmoid(x);
  }
}

// The derivative.  Where the factor beside sigma*(1 - sigma) could overflow
// while that product is 0, it is bounded (a NaN of x arrives through sigma).
template <int ACT>
__device__ __forceinline__ float act_slope(float x) {
  float s, ds;
  if constexpr (ACT == kActGelu) {
    normal_cdf(x, s, ds);
    return __builtin_fmaf(x * 0.39894228040143268f, ds, s);
  } else if constexpr (ACT == kActGeluTanh) {
    sigmoid_slope(kGeluC * x * __builtin_fmaf(kGeluK * x, x, 1.0f), s, ds);
    const float c = __builtin_amdgcn_fmed3f(x, -64.0f, 64.0f);
    return __builtin_fmaf(ds, kGeluC * c * __builtin_fmaf(3.0f * kGeluK * c, c, 1.0f), s);
  } else {
    sigmoid_slope(x, s, ds);
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

// This wavefront's tile: first column of the lane, its first row, its number
// of columns; false where nothing is left to do.
struct Place {
  int64_t row;
  int col;
  int n;
  int64_t block;
};

__device__ __forceinline__ bool place(const ActArgs &a, Place &at) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x * kWaves + wave;
  if (tile >= a.tiles) return false;
  const uint32_t blk = tile / a.col_tiles, ct = tile - blk * a.col_tiles;
  const int lane = threadIdx.x & 63;
  at.block = blk;
  at.row = static_cast<int64_t>(blk) * kActBlock + (lane >> 4);
  at.col = static_cast<int>(ct) * kCols + (lane & 15) * 8;
  at.n = static_cast<int>(a.cols - at.col);
  return true;
}

template <typename T, int FMT, int ACT, bool VEC>
__global__ __launch_bounds__(kBlock) void act_save_kernel(const ActArgs a) {
  Place at;
  if (!place(a, at)) return;
  float v[kRowsPerLane][8];
#pragma unroll
  for (int j = 0; j < kRowsPerLane; ++j) {
    const int64_t r = at.row + 4 * j;
    load8<T, VEC>(static_cast<const T *>(a.x) + r * a.ldx + at.col, r < a.rows ? at.n : 0, v[j]);
  }
  uint32_t scale[8];
  float inv[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kRowsPerLane; ++j) m = max(m, __float_as_uint(v[j][k]) & 0x7fffffffu);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
    scale[k] = act_scale<FMT>(m);
    // a NaN block: NaN * x encodes as the NaN code of e4m3; int8 codes are 0 there
    inv[k] = scale[k] == kNanScale ? (FMT == kE4M3 ? __uint_as_float(0x7fc00000u) : 0.0f)
                                   : __uint_as_float((254u - scale[k]) << 23);
  }
  if (at.n <= 0) return;
  uint8_t *codes = a.codes + at.col;
#pragma unroll
  for (int j = 0; j < kRowsPerLane; ++j) {
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
      for (int k = 0; k < 8; ++k) y[k] = act_value<ACT>(v[j][k]);
      store8<T, VEC>(static_cast<T *>(a.y) + r * a.ldy + at.col, at.n, y);
    }
  }
  if ((threadIdx.x & 48) == 0) {
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
  if (!place(a, at) || at.n <= 0) return;
  float s[8];
  load_scales<FMT>(a, at, s);
  u32x2 w[kRowsPerLane];
#pragma unroll
  for (int j = 0; j < kRowsPerLane; ++j) {
    const int64_t r = at.row + 4 * j;
    w[j] = u32x2{0, 0};
    if (r < a.rows) w[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(a.codes_in + r * a.pitch + at.col));
  }
  float g[kRowsPerLane][8];
  if constexpr (ACT != kActNone) {
#pragma unroll
    for (int j = 0; j < kRowsPerLane; ++j) {
      const int64_t r = at.row + 4 * j;
      load8<T, VEC>(static_cast<const T *>(a.x) + r * a.ldx + at.col, r < a.rows ? at.n : 0, g[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kRowsPerLane; ++j) {
    const int64_t r = at.row + 4 * j;
    if (r >= a.rows) break;
    __builtin_amdgcn_sched_barrier(0);    // a row at a time: decoding all rows first takes registers for nothing
    float x[8];
    decode8<FMT>(w[j], s, x);
    if constexpr (ACT != kActNone) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = g[j][k] * act_slope<ACT>(x[k]);
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
void save_one(const ActArgs &a, dim3 grid, hipStream_t s) {
  if (vector_rows(a, sizeof(T))) act_save_kernel<T, FMT, ACT, true><<<grid, kBlock, 0, s>>>(a);
  else act_save_kernel<T, FMT, ACT, false><<<grid, kBlock, 0, s>>>(a);
}

template <typename T, int FMT, int ACT>
void read_one(const ActArgs &a, dim3 grid, hipStream_t s) {
  if (vector_rows(a, sizeof(T))) act_read_kernel<T, FMT, ACT, true><<<grid, kBlock, 0, s>>>(a);
  else act_read_kernel<T, FMT, ACT, false><<<grid, kBlock, 0, s>>>(a);
}

template <typename T, int FMT>
void by_act(bool save, int act, const ActArgs &a, dim3 grid, hipStream_t s) {
  if (save) {
    if (act == kActGelu) save_one<T, FMT, kActGelu>(a, grid, s);
    else if (act == kActGeluTanh) save_one<T, FMT, kActGeluTanh>(a, grid, s);
    else if (act == kActSilu) save_one<T, FMT, kActSilu>(a, grid, s);
    else save_one<T, FMT, kActNone>(a, grid, s);
  } else {
    if (act == kActGelu) read_one<T, FMT, kActGelu>(a, grid, s);
    else if (act == kActGeluTanh) read_one<T, FMT, kActGeluTanh>(a, grid, s);
    else if (act == kActSilu) read_one<T, FMT, kActSilu>(a, grid, s);
    else read_one<T, FMT, kActNone>(a, grid, s);
  }
}

}  // namespace

int64_t act_tiles(int64_t rows, int64_t cols) {
  return act_blocks(rows) * ((cols + kCols - 1) / kCols);
}

void launch_act(bool save, int fmt, int act, bool bf16, ActArgs a, hipStream_t s) {
  a.col_tiles = static_cast<uint32_t>((a.cols + kCols - 1) / kCols);
  a.tiles = static_cast<uint32_t>(act_tiles(a.rows, a.cols));
  a.pitch = act_pitch(a.cols);
  const dim3 grid((a.tiles + kWaves - 1) / kWaves);
  if (bf16) {
    if (fmt == kE4M3) by_act<uint16_t, kE4M3>(save, act, a, grid, s);
    else by_act<uint16_t, kInt8>(save, act, a, grid, s);
  } else {
    if (fmt == kE4M3) by_act<float, kE4M3>(save, act, a, grid, s);
    else by_act<float, kInt8>(save, act, a, grid, s);
  }
}

}  // namespace ob
