// AdamW over the whole list in one pass (gfx950), with its moments as fp32 or
// in 8 bits, and the 8-bit moments' values.
//
//   g = (sum over w ascending of g_w) / W (* grad_scale)
//   m = c1 m + c2 g;   v = b2 v + cb2 (g g);   r = sqrt(v)
//   p = (p - p k_t) - (m / (r root + eps)) step,   k_t = fp32(lr wd) * decay_t
// every fp32 operation rounded once.  A chunk of 1024 elements of one tensor is
// a workgroup's, four consecutive elements a lane's, so every fp32 row is read
// and written in 16-byte vectors and 16 lanes (one DPP row) hold a block of 64.
//
// 8-bit moments.  64 consecutive elements of the list share a scale byte s,
// 2^(s - 127), the smallest power of two (at least 2^-111) for which the block's
// largest magnitude fits.  m is held as e4m3; of v its root, as an unsigned float
// of 4 exponent and 4 mantissa bits (code c = 16 k + f: f for k = 0, else
// (16 + f) 2^(k-1)): the root halves the exponent range that v needs.
//
// Rounding.  To the nearest code v would stop: with beta2 = 0.999 a step moves
// it by a thousandth, a code's half step is a thirtieth, so v stayed at a quarter
// of its true value while gradients grew and at six times it after they fell
// tenfold (simulated over 6000 steps).  So codes are rounded down or up with the
// probability of the remainder in 16 bits: unbiased to within 2^-16 of a step (v's
// median within 5% over the same steps, 90% of the elements within a factor of 1.5 to 2).  The 16 bits that
// settle it are a hash of the element's place and the caller's seed, so a step
// repeats bit for bit.  Where x is scaled so that the format's subnormal codes
// lie at fp32's, adding them below the code's last bit and cutting off the rest
// is this rounding, carry into the exponent and subnormals included.
// A root above 0 keeps the smallest code at least: 0 under a moment that is not 0
// would make the step m/eps.
//
// Bound by the memory: gradients are streamed past the caches, eight workers' rows
// loaded four at a time before they are added.  Eight workers of fp32 gradients with
// fp32 moments and a bf16 copy of the weights (107 M elements, 6.2 GB) 1145 us, 5.4 TB/s;
// one worker's bf16 gradients with 8-bit moments (334 M, 5.4 GB) 975-1020 us, 5.3-5.6; their
// values read back as bf16 (2.1 GB) 393-401 us.  Small lists are the launch's: 2050
// elements 3 us, 1.8 M with 8-bit moments 10.
#include "internal.h"
#include "activation.h"

#pragma clang fp contract(off)

namespace ob {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

constexpr int kQuadBlock = 16;          // lanes of a block of kMomentBlock elements
static_assert(kQuadBlock * 4 == kMomentBlock && kChunk == kBlock * 4, "four elements a lane");

// Up to four elements from p on; absent ones are 0.
template <bool FULL, bool STREAM>
__device__ __forceinline__ f32x4 load4(const float *p, int n) {
  if (FULL || n >= 4) {
    if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
    return *reinterpret_cast<const f32x4 *>(p);
  }
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < n) v[k] = p[k];
  return v;
}

template <bool FULL, bool STREAM>
__device__ __forceinline__ f32x4 load4(const uint16_t *p, int n) {
  uint32_t h[4] = {0, 0, 0, 0};
  if (FULL || n >= 4) {
    const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p));
    h[0] = w[0] << 16;
    h[1] = w[0] & 0xffff0000u;
    h[2] = w[1] << 16;
    h[3] = w[1] & 0xffff0000u;
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < n) h[k] = static_cast<uint32_t>(p[k]) << 16;
  }
  f32x4 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(h[k]);
  return v;
}

// Four bytes, the first in the lowest bits; absent ones are 0.
template <bool FULL>
__device__ __forceinline__ uint32_t load_codes(const uint8_t *p, int n) {
  if (FULL || n >= 4) return *reinterpret_cast<const uint32_t *>(p);
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < n) w |= static_cast<uint32_t>(p[k]) << (8 * k);
  return w;
}

template <bool FULL>
__device__ __forceinline__ void store_codes(uint8_t *p, int n, uint32_t w) {
  if (FULL || n >= 4) {
    *reinterpret_cast<uint32_t *>(p) = w;
    return;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < n) p[k] = static_cast<uint8_t>(w >> (8 * k));
}

template <bool FULL>
__device__ __forceinline__ void store4(float *p, int n, f32x4 v) {
  if (FULL || n >= 4) {
    *reinterpret_cast<f32x4 *>(p) = v;
    return;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < n) p[k] = v[k];
}

// Rounded to bf16, to the nearest and halves to even.
template <bool FULL>
__device__ __forceinline__ void store4(uint16_t *p, int n, f32x4 v) {
  uint16_t h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[k]));
  if (FULL || n >= 4) {
    u32x2 w;
    w[0] = h[0] | static_cast<uint32_t>(h[1]) << 16;
    w[1] = h[2] | static_cast<uint32_t>(h[3]) << 16;
    *reinterpret_cast<u32x2 *>(p) = w;
    return;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < n) p[k] = h[k];
}

// Largest of the 16 lanes of a DPP row.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xf, 0xf, true)));    // quad_perm 1,0,3,2
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xf, 0xf, true)));    // quad_perm 2,3,0,1
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x141, 0xf, 0xf, true)));   // the half row reversed
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x140, 0xf, 0xf, true)));  // the row reversed
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The scale byte of a block of roots from its largest bit pattern: 31 * 2^14,
// the largest code, is 1.9375 * 2^18.
__device__ __forceinline__ uint32_t root_scale(uint32_t amax) {
  if (amax >= kInfBits) return kNanScale;
  const uint32_t p = (amax + 0x07ffffu) >> 23;
  return p < kMinScale + 18u ? kMinScale : p - 18u;
}

// 2^-(s - 127), for s up to 254.
__device__ __forceinline__ float inverse_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }

__device__ __forceinline__ f32x4 decode_m(uint32_t w, float scale) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
  const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
  return f32x4{lo[0] * scale, lo[1] * scale, hi[0] * scale, hi[1] * scale};
}

// Roots: a code's bits below an fp32 exponent field are its value * 2^-130.
__device__ __forceinline__ f32x4 decode_root(uint32_t w, float scale) {
  const float up = scale * 0x1p65f;
  f32x4 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = (__uint_as_float(((w >> (8 * k)) & 0xffu) << 19) * 0x1p65f) * up;
  return r;
}

// The codes of four moments and their block's scale byte; d: 16 bits each.
__device__ __forceinline__ uint32_t encode_m(f32x4 m, const uint32_t (&d)[4], uint32_t &s) {
  uint32_t a = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) a = max(a, magnitude(m[k]));
  s = act_scale<kE4M3>(row_max(a));
  if (s == kNanScale) return 0;
  const float down = inverse_scale(s);
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float t = (__uint_as_float(min(magnitude(m[k]), kTopBits)) * down) * 0x1p-120f;
    const uint32_t code = (__float_as_uint(t) + (d[k] << 4)) >> 20;
    w |= (code | (__float_as_uint(m[k]) >> 31) << 7) << (8 * k);
  }
  return w;
}

__device__ __forceinline__ uint32_t encode_root(f32x4 r, const uint32_t (&d)[4], uint32_t &s) {
  uint32_t a = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) a = max(a, magnitude(r[k]));
  s = root_scale(row_max(a));
  if (s == kNanScale) return 0;
  const float down = inverse_scale(s);
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float t = ((r[k] * down) * 0x1p-65f) * 0x1p-65f;
    const uint32_t code = (__float_as_uint(t) + (d[k] << 3)) >> 19;
    w |= max(code, r[k] > 0.0f ? 1u : 0u) << (8 * k);
  }
  return w;
}

template <typename G, bool EIGHT, bool FULL>
__device__ __forceinline__ void adamw_chunk(const Tile &tl, int sub0, const Geometry &g, const AdamwArgs &a) {
  const int at = sub0 + static_cast<int>(threadIdx.x) * 4;
  const int n = FULL ? 4 : min(4, tl.len - at);       // this lane's elements, none if below 1
  const int64_t i = tl.start + at;
  constexpr int kGroup = 4;                           // workers whose loads are under way together
  const G *grads = static_cast<const G *>(a.grads) + i;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 m, v;
  uint32_t mw = 0, vw = 0, ms = 0, vs = 0;
  if constexpr (EIGHT) {
    if (FULL || n > 0) {
      mw = load_codes<FULL>(static_cast<const uint8_t *>(a.m) + i, n);
      vw = load_codes<FULL>(static_cast<const uint8_t *>(a.v) + i, n);
      ms = a.m_scale[i / kMomentBlock];
      vs = a.v_scale[i / kMomentBlock];
    }
  } else {
    m = load4<FULL, false>(static_cast<const float *>(a.m) + i, n);
    v = load4<FULL, false>(static_cast<const float *>(a.v) + i, n);
  }
  f32x4 p = load4<FULL, false>(a.params + i, n);
  for (int w0 = 0; w0 < g.W; w0 += kGroup) {
    f32x4 x[kGroup];
#pragma unroll
    for (int k = 0; k < kGroup; ++k)
      if (w0 + k < g.W) x[k] = load4<FULL, true>(grads + static_cast<size_t>(w0 + k) * g.N, n);
#pragma unroll
    for (int k = 0; k < kGroup; ++k)
      if (w0 + k < g.W) acc += x[k];
  }
  const float wf = static_cast<float>(g.W), inv_w = 1.0f / wf;
  const bool pow2 = (g.W & (g.W - 1)) == 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = pow2 ? acc[k] * inv_w : acc[k] / wf;
  if (a.grad_scale) {
    const float gs = *a.grad_scale;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = acc[k] * gs;
  }
  if constexpr (EIGHT) {
    m = decode_m(mw, act_scale_value(ms));
    v = decode_root(vw, act_scale_value(vs));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = v[k] * v[k];
  }
  const float fade = a.decay ? a.fade * a.decay[tl.tensor] : a.fade;
  f32x4 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    m[k] = a.c1 * m[k] + a.c2 * acc[k];
    v[k] = a.b2 * v[k] + a.cb2 * (acc[k] * acc[k]);
    r[k] = __builtin_sqrtf(v[k]);
    const float u = m[k] / (r[k] * a.root + a.eps);
    p[k] = (p[k] - p[k] * fade) - u * a.step;
  }
  if constexpr (EIGHT) {
    if (!FULL) {     // absent elements are no part of their block
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k >= n) m[k] = r[k] = 0.0f;
    }
    const uint32_t key = a.key + static_cast<uint32_t>(static_cast<uint64_t>(i) >> 32) * 0x9E3779B9u;
    uint32_t dm[4], dv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t h = mix32((static_cast<uint32_t>(i) + k) ^ key);
      dm[k] = h & 0xffffu;
      dv[k] = h >> 16;
    }
    mw = encode_m(m, dm, ms);
    vw = encode_root(r, dv, vs);
    if (FULL || n > 0) {
      store_codes<FULL>(static_cast<uint8_t *>(a.m) + i, n, mw);
      store_codes<FULL>(static_cast<uint8_t *>(a.v) + i, n, vw);
      if (threadIdx.x % kQuadBlock == 0) {
        a.m_scale[i / kMomentBlock] = static_cast<uint8_t>(ms);
        a.v_scale[i / kMomentBlock] = static_cast<uint8_t>(vs);
      }
    }
  } else {
    store4<FULL>(static_cast<float *>(a.m) + i, n, m);
    store4<FULL>(static_cast<float *>(a.v) + i, n, v);
  }
  store4<FULL>(a.params + i, n, p);
  if (a.model) store4<FULL>(a.model + i, n, p);
}

template <typename G, bool EIGHT>
__global__ __launch_bounds__(kBlock) void adamw_kernel(Geometry g, AdamwArgs a) {
  const Tile tl = g.tiles[blockIdx.x / kChunksPerTile];
  const int sub0 = static_cast<int>(blockIdx.x % kChunksPerTile) * kChunk, rem = tl.len - sub0;
  if (rem <= 0) return;
  if (rem >= kChunk) adamw_chunk<G, EIGHT, true>(tl, sub0, g, a);
  else adamw_chunk<G, EIGHT, false>(tl, sub0, g, a);
}

// The 8-bit moments' values, in chunks as above.
template <typename T, bool FULL>
__device__ __forceinline__ void load_chunk(const Tile &tl, int sub0, const AdamwArgs &a, T *m, T *v) {
  const int at = sub0 + static_cast<int>(threadIdx.x) * 4;
  const int n = FULL ? 4 : min(4, tl.len - at);
  if (!FULL && n <= 0) return;
  const int64_t i = tl.start + at;
  const uint32_t mw = load_codes<FULL>(static_cast<const uint8_t *>(a.m) + i, n);
  const uint32_t vw = load_codes<FULL>(static_cast<const uint8_t *>(a.v) + i, n);
  const f32x4 x = decode_m(mw, act_scale_value(a.m_scale[i / kMomentBlock]));
  f32x4 y = decode_root(vw, act_scale_value(a.v_scale[i / kMomentBlock]));
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] = y[k] * y[k];
  store4<FULL>(m + i, n, x);
  store4<FULL>(v + i, n, y);
}

template <typename T>
__global__ __launch_bounds__(kBlock) void adamw_load_kernel(Geometry g, AdamwArgs a, T *m, T *v) {
  const Tile tl = g.tiles[blockIdx.x / kChunksPerTile];
  const int sub0 = static_cast<int>(blockIdx.x % kChunksPerTile) * kChunk, rem = tl.len - sub0;
  if (rem <= 0) return;
  if (rem >= kChunk) load_chunk<T, true>(tl, sub0, a, m, v);
  else load_chunk<T, false>(tl, sub0, a, m, v);
}

}  // namespace

void launch_adamw(const Geometry &g, bool bf16, bool eight, const AdamwArgs &a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(g.num_tiles) * kChunksPerTile));   // at most kMaxGrid
  if (bf16) {
    if (eight) adamw_kernel<uint16_t, true><<<grid, kBlock, 0, s>>>(g, a);
    else adamw_kernel<uint16_t, false><<<grid, kBlock, 0, s>>>(g, a);
  } else {
    if (eight) adamw_kernel<float, true><<<grid, kBlock, 0, s>>>(g, a);
    else adamw_kernel<float, false><<<grid, kBlock, 0, s>>>(g, a);
  }
}

void launch_adamw_load(const Geometry &g, const AdamwArgs &a, bool bf16, void *m, void *v, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(g.num_tiles) * kChunksPerTile));
  if (bf16) adamw_load_kernel<<<grid, kBlock, 0, s>>>(g, a, static_cast<uint16_t *>(m), static_cast<uint16_t *>(v));
  else adamw_load_kernel<<<grid, kBlock, 0, s>>>(g, a, static_cast<float *>(m), static_cast<float *>(v));
}

}  // namespace ob
