// Device helpers of the kernels that multiply matrices (linear_grad.hip,
// linear.hip): tiles that go from memory straight to LDS, and the workgroups'
// order.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace ob {

#define OB_LDS __attribute__((address_space(3)))

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(2))) int i32x2;
typedef __attribute__((ext_vector_type(4))) int i32x4;

// Rows of a tile are spread over the LDS banks by an exclusive or on the
// 32-byte unit within the row, so that the rows one transposing read touches lie
// on different banks.
__device__ __forceinline__ int swizzle_a(int r) { return (r & 3) | ((r >> 3) & 1) << 2; }
// A buffer of `bytes` from `base` on: reads past its end give 0, which is what
// missing tokens contribute.  Its end is rounded up to the 16 bytes that one
// load takes (all loads start on 16 bytes, so such a load stays within memory
// that the matrix's last element lies in; what it reads there belongs to
// columns that are dropped).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (bytes + 15) & ~15, 0x00020000);
}

// Start the copy of 16 or 4 bytes a lane, from its own offset, to LDS in lane
// order.
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t from, OB_LDS unsigned char *to, int offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (OB_LDS void *)to, 16, offset, 0, 0, 0);
}

__device__ __forceinline__ void copy4(__amdgpu_buffer_rsrc_t from, OB_LDS unsigned char *to, int offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (OB_LDS void *)to, 4, offset, 0, 0, 0);
}

// A workgroup's place: consecutive workgroups go to the 8 XCDs in turn, so
// the tiles are numbered such that each XCD (its own L2) gets a consecutive
// range: one slice of the contraction where there are several, and within it
// kGroup tiles along the first side times a run along the second, the shape that
// needs the fewest bytes of both.
constexpr int kXcds = 8, kGroup = 4;
struct Split {
  int m_tiles, n_tiles;
  int splits;                // slices of the contraction; more than one: joined from the workspace
  int64_t turns_each;
};
struct Where {
  int mt, nt, split;
};
__device__ __forceinline__ Where where(const Split &sp) {
  const uint32_t m_tiles = sp.m_tiles, n_tiles = sp.n_tiles;
  const uint32_t tiles = m_tiles * n_tiles, total = tiles * sp.splits;
  const uint32_t id = blockIdx.x, xcd = id % kXcds, at = id / kXcds;
  const uint32_t each = total / kXcds, more = total % kXcds;
  const uint32_t lin = xcd * each + min(xcd, more) + at;
  const uint32_t split = lin / tiles, t = lin - split * tiles;
  const uint32_t band = t / (kGroup * n_tiles), in_band = t - band * kGroup * n_tiles;
  const uint32_t high = min(uint32_t{kGroup}, m_tiles - band * kGroup);
  // uniform over the workgroup: kept in scalar registers
  return Where{__builtin_amdgcn_readfirstlane(static_cast<int>(band * kGroup + in_band % high)),
               __builtin_amdgcn_readfirstlane(static_cast<int>(in_band / high)), __builtin_amdgcn_readfirstlane(static_cast<int>(split))};
}

// Waits until at most N of this wavefront's loads are out and its LDS accesses
// are done.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

}  // namespace ob
