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
#include "internal.h"
#include "activation.h"
#include "act_math.h"

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
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

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
    inv[k] = act_inverse<FMT>(scale[k]);
  }
  if (at.n <= 0) return;
  uint8_t *codes = a.codes + at.col;
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t r = at.row + 4 * j;
    if (r >= a.rows) break;
    const u32x2 w = encode8<FMT>(v[j], inv);
    uint8_t *out = codes + r * a.pitch;
    if (at.n >= 8) {
      *reinterpret_cast<u32x2 *>(out) = w;
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
    s[k] = act_scale_or_nan(b);
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
