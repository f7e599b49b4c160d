// The 8-bit activation checkpoint: its format and the device helpers that
// encode and decode it, shared by activation.hip (save, load, activation
// backward) and linear_grad.hip (weight gradient).
//
// Format.  x is [rows][cols].  kActBlock consecutive rows of one column share
// one scale byte s, standing for the scale 2^(s - 127).  Codes are bytes,
// [rows][pitch] with pitch = 64*ceil(cols/64); scales are bytes,
// [ceil(rows/32)][pitch].  With a = max|x| over a block and p = floor(log2 a):
//   e4m3  s - 127 = p - 8, one more if a > 1.75 * 2^p  (a / 2^(s-127) <= 448)
//   int8  s - 127 = p - 6, one more if a > 127 * 2^(p-6)  (a / 2^(s-127) <= 127)
// and at least -111; magnitudes past 1.875 * 2^127 count as that (rounding
// them up would leave the range of floats); code = x / 2^(s-127), rounded to nearest even.  Scaling
// by a power of two is exact, so the code's rounding is the only one, and
// because a code has at most 7 significant bits and the scale is at least
// 2^-111, the decoded value is exact in bf16.  A block with a NaN or an
// infinity has s = 255 and reads as NaN throughout.
//
// Why along rows (tokens): large activations sit in a few feature columns for
// all tokens, so a block of one column keeps them from widening the steps of
// their neighbours; and the weight gradient contracts over tokens, so the 32
// contraction steps of one 16x16x32 matrix instruction share one scale per
// lane.  The power-of-two scale costs at most one bit of an int8 code.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace ob {

constexpr int kActBlock = 32;
constexpr int kE4M3 = 0, kInt8 = 1;               // OB_ACT_E4M3, OB_ACT_INT8
constexpr uint32_t kMinScale = 16;                // 2^-111
constexpr uint32_t kNanScale = 255;
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kTopBits = 0x7f700000u;        // 1.875 * 2^127

__host__ __device__ inline int64_t act_pitch(int64_t cols) { return (cols + 63) / 64 * 64; }
__host__ __device__ inline int64_t act_blocks(int64_t rows) { return (rows + kActBlock - 1) / kActBlock; }

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;

// The scale byte of a block from the largest |x| bit pattern in it: as
// unsigned integers these order like the magnitudes, infinities and NaNs on
// top.  Adding the distance from the mantissa's limit to the next power of
// two carries into the exponent exactly when the largest code would be
// passed.
template <int FMT>
__device__ __forceinline__ uint32_t act_scale(uint32_t amax) {
  if (amax >= kInfBits) return kNanScale;
  const uint32_t p = (min(amax, kTopBits) + (FMT == kE4M3 ? 0x1fffffu : 0x01ffffu)) >> 23;
  const uint32_t top = FMT == kE4M3 ? 8u : 6u;
  return p < kMinScale + top ? kMinScale : p - top;
}

// The fp32 scale of a scale byte.  255 gives an infinity: the e4m3 conversion
// makes every element a NaN with it, and int8 codes are 0 in such a block, so
// their product with it is a NaN too.
__device__ __forceinline__ float act_scale_value(uint32_t s) { return __uint_as_float(s << 23); }

// Two decoded values (bytes 2h and 2h+1 of w) with one scale, as bf16; exact.
template <int FMT, bool HIGH>
__device__ __forceinline__ bf16x2 act_decode2(uint32_t w, float scale) {
  if constexpr (FMT == kE4M3) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HIGH);
  } else {
    const int v = static_cast<int>(HIGH ? w : w << 16);
    const float lo = static_cast<float>(static_cast<int8_t>(v >> 16)) * scale;
    const float hi = static_cast<float>(v >> 24) * scale;
    bf16x2 r;
    r[0] = static_cast<__bf16>(lo);
    r[1] = static_cast<__bf16>(hi);
    return r;
  }
}

}  // namespace ob
