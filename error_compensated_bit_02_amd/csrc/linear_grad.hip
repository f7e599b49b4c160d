// Weight and bias gradient of a linear layer from an 8-bit checkpoint of its
// input (gfx950):
//   dW[o][i] = sum over t of dY[t][o] * X[t][i],   db[o] = sum over t of dY[t][o]
// with X the checkpoint's values.  The result goes straight into one worker's
// gradient row of the tensor list.
//
// The contraction runs on the bf16 matrix units with fp32 accumulators.  X is
// exact in bf16 (activation.h), so with bf16 dY the products are exact.  An
// fp32 dY is cut into three bf16 parts of 8 significant bits each, which add
// up to it exactly; three products per element keep fp32 accuracy at a third
// of the bf16 rate.
//
// Both operands lie with the contraction index t slowest ([t][o] and [t][i]),
// and a matrix instruction wants 8 consecutive t per lane: the tiles go to LDS
// as they are and come back transposed (ds_read_b64_tr_b16 for dY,
// ds_read_b64_tr_b8 for the codes).  The codes stay bytes in LDS and are
// converted after the read, one scale per lane and 32 tokens.  X is the
// instruction's first operand, so a lane's four results are four consecutive
// i of one weight row, stored as one vector.
#include "internal.h"
#include "activation.h"

#pragma clang fp contract(off)

namespace ob {
namespace {

#define OB_LDS __attribute__((address_space(3)))

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(2))) int i32x2;
typedef __attribute__((ext_vector_type(4))) int i32x4;

// Rows of a tile are spread over the LDS banks by an exclusive or on the
// 32-byte (dY) or 16-byte (codes) unit within the row, so that the rows one
// transposing read touches lie on different banks.
__device__ __forceinline__ int swizzle_a(int r) { return (r & 3) | ((r >> 3) & 1) << 2; }
template <int BN>
__device__ __forceinline__ int swizzle_b(int r) {
  return BN >= 256 ? ((r & 7) | ((r >> 3) & 1) << 3) : (r & 7);
}

// A buffer over what is left of a matrix from byte0 on: reads past its end
// give 0, which is what the missing tokens contribute.  The end is rounded up
// to the 16 bytes that one load takes (all loads start on 16 bytes, so such a
// load stays within memory that the matrix's last element lies in; what it
// reads there belongs to columns that are dropped).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rest(const void *base, int64_t byte0, int64_t bytes) {
  int64_t left = (bytes + 15) / 16 * 16 - byte0;
  left = left < 0 ? 0 : left > 0x7fffffff ? 0x7fffffff : left;
  return __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char *>(static_cast<const char *>(base) + (left ? byte0 : 0)), 0, static_cast<int>(left), 0x00020000);
}

// An fp32 value as three bf16 parts (truncated, so no part overflows).
__device__ __forceinline__ void split3(float x, uint32_t &h, uint32_t &m, uint32_t &l) {
  const uint32_t b = __float_as_uint(x);
  h = b >> 16;
  const float r1 = (b & 0x7fffffffu) == kInfBits ? 0.0f : x - __uint_as_float(b & 0xffff0000u);
  const uint32_t b1 = __float_as_uint(r1);
  m = b1 >> 16;
  const float r2 = r1 - __uint_as_float(b1 & 0xffff0000u);
  l = __float_as_uint(r2) >> 16;
}

// Writes a wavefront's results: to `part`, a matrix of its own, or rounded
// into the gradient.  Lane: weight row lane % 16 of a fragment, four
// consecutive columns.
template <int BM, int BN, int WM, int WN, int FO, int FI>
__device__ __forceinline__ void store_tile(const LinearArgs &a, const f32x4 (&acc)[FI][FO], int64_t m0, int64_t n0, int wm,
                                           int wn, float *part) {
  const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
  const bool quad = a.in % 4 == 0;
#pragma unroll
  for (int o = 0; o < FO; ++o) {
    const int64_t row = m0 + (wm * FO + o) * 16 + li;
    if (row >= a.out) continue;
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      const int64_t col = n0 + (wn * FI + i) * 16 + g * 4;
      if (col >= a.in) continue;
      const int64_t at = row * a.in + col;
      f32x4 v = acc[i][o];
      if (part) {
        float *p = part + at;
        if (quad) {
          *reinterpret_cast<f32x4 *>(p) = v;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (col + k < a.in) p[k] = v[k];
        }
      } else if (a.grad_bf16) {
        uint16_t *p = static_cast<uint16_t *>(a.dw) + at;
        uint16_t r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (col + k < a.in) {
            if (a.accumulate) v[k] += __uint_as_float(static_cast<uint32_t>(p[k]) << 16);
            r[k] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[k]));
          }
        }
        if (quad) {
          __builtin_memcpy(__builtin_assume_aligned(p, 8), r, 8);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (col + k < a.in) p[k] = r[k];
        }
      } else {
        float *p = static_cast<float *>(a.dw) + at;
        if (quad) {
          if (a.accumulate) v += *reinterpret_cast<const f32x4 *>(p);
          *reinterpret_cast<f32x4 *>(p) = v;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (col + k < a.in) p[k] = a.accumulate ? p[k] + v[k] : v[k];
        }
      }
    }
  }
}

// BM x BN tile of dW, WM x WN wavefronts, BK tokens a turn.  PARTS: bf16 parts
// of dY (1: bf16, 3: fp32).  VEC: 16-byte loads of dY (its rows start on 16
// bytes and a turn's rows lie within 2 GB).
template <int BM, int BN, int BK, int WM, int WN, int PARTS, int FMT, bool VEC>
__global__ __launch_bounds__(64 * WM * WN) void linear_grad_kernel(const LinearArgs a, int m_tiles, int n_tiles,
                                                          int64_t turns_each, float *part) {
  constexpr int NT = 64 * WM * WN;
  constexpr int FO = BM / WM / 16, FI = BN / WN / 16;   // 16-wide fragments of a wavefront
  constexpr int A_BYTES = BK * BM * 2, B_BYTES = BK * BN, S_BYTES = BK / 32 * BN;
  constexpr int STAGE = PARTS * A_BYTES + B_BYTES + S_BYTES;
  constexpr int CA = BM / 8, RA = NT / CA, JA = BK / RA;     // dY: 8-element chunks a row, rows a step, steps
  constexpr int CB = BN / 16, RB = NT / CB, JB = BK / RB;    // codes: 16-byte chunks
  constexpr int JS = (S_BYTES + NT - 1) / NT;
  static_assert(JA >= 1 && JB >= 1 && BK % RA == 0 && BK % RB == 0, "tile too small");
  __shared__ __attribute__((aligned(1024))) unsigned char lds[2 * STAGE];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN;
  const int tile = blockIdx.x;
  const int nt = tile % n_tiles, mt = tile / n_tiles;
  const int64_t m0 = static_cast<int64_t>(mt) * BM, n0 = static_cast<int64_t>(nt) * BN;
  const int64_t turn0 = blockIdx.y * turns_each;
  const int64_t all = (a.rows + BK - 1) / BK;
  const int64_t turns = max(int64_t{0}, min(turns_each, all - turn0));

  f32x4 acc[FI][FO];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int o = 0; o < FO; ++o) acc[i][o] = f32x4{0, 0, 0, 0};

  // staging registers: one turn's dY, codes and scales
  constexpr int ES = PARTS == 1 ? 2 : 4;
  i32x4 ra[JA][ES / 2], rb[JB];
  uint32_t rs[JS];
  const int ca = tid % CA, r_a = tid / CA, cb = tid % CB, r_b = tid / CB;

  auto load = [&](int64_t turn) {
    const int64_t t0 = (turn0 + turn) * BK;
    if constexpr (VEC) {
      const auto rsrc = rest(a.dy, (t0 * a.lddy + m0) * ES, ((a.rows - 1) * a.lddy + a.out) * ES);
#pragma unroll
      for (int j = 0; j < JA; ++j) {
        const int off = static_cast<int>((r_a + RA * j) * a.lddy + ca * 8) * ES;
#pragma unroll
        for (int h = 0; h < ES / 2; ++h) ra[j][h] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, off + 16 * h, 0, 0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < JA; ++j) {
        const int64_t t = t0 + r_a + RA * j, m = m0 + ca * 8;
        const int n = t < a.rows ? static_cast<int>(min(int64_t{8}, a.out - m)) : 0;
        const char *p = static_cast<const char *>(a.dy) + (t * a.lddy + m) * ES;
        if (n == 8) {
          __builtin_memcpy(&ra[j][0], p, 8 * ES);
        } else {
          uint32_t w[2 * ES];
#pragma unroll
          for (int k = 0; k < 2 * ES; ++k) w[k] = 0;
#pragma unroll
          for (int k = 0; k < 7; ++k) {
            if (k < n) {
              if constexpr (ES == 4) w[k] = reinterpret_cast<const uint32_t *>(p)[k];
              else w[k >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[k]) << (16 * (k & 1));
            }
          }
#pragma unroll
          for (int k = 0; k < 2 * ES; ++k) ra[j][k >> 2][k & 3] = static_cast<int>(w[k]);
        }
      }
    }
    const auto crsrc = rest(a.codes, t0 * a.pitch + n0, a.rows * a.pitch);
#pragma unroll
    for (int j = 0; j < JB; ++j)
      rb[j] = __builtin_amdgcn_raw_buffer_load_b128(crsrc, static_cast<int>((r_b + RB * j) * a.pitch) + cb * 16, 0, 0);
    const auto srsrc = rest(a.scales, t0 / kActBlock * a.pitch + n0, act_blocks(a.rows) * a.pitch);
#pragma unroll
    for (int j = 0; j < JS; ++j) {
      const int at = tid + NT * j;
      rs[j] = at >= S_BYTES ? 0u : __builtin_amdgcn_raw_buffer_load_b8(srsrc, static_cast<int>(at / BN * a.pitch) + at % BN, 0, 0);
    }
  };

  auto store = [&](int buf) {
    unsigned char *A = lds + buf * STAGE, *B = A + PARTS * A_BYTES, *S = B + B_BYTES;
#pragma unroll
    for (int j = 0; j < JA; ++j) {
      const int r = r_a + RA * j;
      unsigned char *p = A + r * (BM * 2) + (((ca >> 1) ^ swizzle_a(r)) << 5) + (ca & 1) * 16;
      if constexpr (PARTS == 1) {
        *reinterpret_cast<i32x4 *>(p) = ra[j][0];
      } else {
        i32x4 w[3];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t h0, m0_, l0, h1, m1, l1;
          split3(__int_as_float(ra[j][k >> 1][(2 * k) & 3]), h0, m0_, l0);
          split3(__int_as_float(ra[j][k >> 1][(2 * k + 1) & 3]), h1, m1, l1);
          w[0][k] = static_cast<int>(h0 | h1 << 16);
          w[1][k] = static_cast<int>(m0_ | m1 << 16);
          w[2][k] = static_cast<int>(l0 | l1 << 16);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<i32x4 *>(p + q * A_BYTES) = w[q];
      }
    }
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      const int r = r_b + RB * j;
      *reinterpret_cast<i32x4 *>(B + r * BN + ((cb ^ swizzle_b<BN>(r)) << 4)) = rb[j];
    }
    // scales: [block][column % 16][column / 16], so a lane's fragments are adjacent
#pragma unroll
    for (int j = 0; j < JS; ++j) {
      const int at = tid + NT * j, col = at % BN;
      if (at < S_BYTES) S[at / BN * BN + (col & 15) * (BN / 16) + (col >> 4)] = static_cast<unsigned char>(rs[j]);
    }
  };

  const int g = lane >> 4, li = lane & 15;
  const int a_row = 8 * g + (li >> 2), a_sw = (li >> 2) | (g & 1) << 2;
  const int b_row = 8 * g + (li >> 1), b_sw = swizzle_b<BN>(b_row);

  // One 32-token step: its operands as they come from LDS, and its products.
  struct Step {
    uint32_t s[FI / 4];
    i32x2 c[FI];
    s16x4 y[PARTS][FO][2];
  };
  auto fetch = [&](int buf, int kk, Step &f) {
    const unsigned char *A = lds + buf * STAGE, *B = A + PARTS * A_BYTES, *S = B + B_BYTES;
#pragma unroll
    for (int q = 0; q < FI / 4; ++q)
      f.s[q] = *reinterpret_cast<const uint32_t *>(S + kk * BN + li * (BN / 16) + wn * FI + 4 * q);
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      const int unit = (wn * FI + i) ^ b_sw;
      f.c[i] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((OB_LDS i32x2 *)(B + (kk * 32 + b_row) * BN + (unit << 4) + (li & 1) * 8));
    }
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
#pragma unroll
      for (int o = 0; o < FO; ++o) {
        const int unit = (wm * FO + o) ^ a_sw;
        const auto *p = A + q * A_BYTES + (kk * 32 + a_row) * (BM * 2) + (unit << 5) + (li & 3) * 8;
        f.y[q][o][0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((OB_LDS s16x4 *)(p));
        f.y[q][o][1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((OB_LDS s16x4 *)(p + 4 * BM * 2));
      }
    }
  };
  auto multiply = [&](const Step &f) {
    bf16x8 x[FI];
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      const float scale = act_scale_value((f.s[i >> 2] >> (8 * (i & 3))) & 0xffu);
      const bf16x2 d[4] = {act_decode2<FMT, false>(f.c[i][0], scale), act_decode2<FMT, true>(f.c[i][0], scale),
                           act_decode2<FMT, false>(f.c[i][1], scale), act_decode2<FMT, true>(f.c[i][1], scale)};
#pragma unroll
      for (int k = 0; k < 8; ++k) x[i][k] = d[k >> 1][k & 1];
    }
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
#pragma unroll
      for (int o = 0; o < FO; ++o) {
        const bf16x8 y = __builtin_bit_cast(bf16x8, __builtin_shufflevector(f.y[q][o][0], f.y[q][o][1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
        for (int i = 0; i < FI; ++i) acc[i][o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], y, acc[i][o], 0, 0, 0);
      }
    }
  };

  // Each step's operands are read one step ahead.  Per turn one barrier, in
  // its last step: behind it the turn's reads are done everywhere and the next
  // turn's tile is in LDS.
  constexpr int KK = BK / 32, UNROLL = KK == 1 ? 2 : 1;
  if (turns > 0) {
    Step f[2];
    load(0);
    store(0);
    if (turns > 1) load(1);
    __syncthreads();
    fetch(0, 0, f[0]);
    for (int64_t it = 0; it < turns; it += UNROLL) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int64_t t = it + u;
        if (t >= turns) break;
        const int buf = static_cast<int>(t & 1);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          constexpr int kBar = 0;
          const int cur = (u * KK + kk) & 1;
          if (kk + 1 < KK) fetch(buf, kk + 1, f[cur ^ 1]);
          if (kk == 0) {
            if (t + 1 < turns) store(buf ^ 1);
            if (t + 2 < turns) load(t + 2);
          }
          if (kk + 1 == KK) {
            __syncthreads();
            if (t + 1 < turns) fetch(buf ^ 1, 0, f[cur ^ 1]);
          }
          __builtin_amdgcn_sched_barrier(kBar);
          multiply(f[cur]);
          __builtin_amdgcn_sched_barrier(kBar);
        }
      }
    }
  }

  store_tile<BM, BN, WM, WN, FO, FI>(a, acc, m0, n0, wm, wn, part ? part + blockIdx.y * a.out * a.in : nullptr);
}

// ---------------------------------------------------------------------------
// The large tile: bf16 dY whose rows start on 16 bytes.
// ---------------------------------------------------------------------------
#define OB_WAIT_VM(n) asm volatile("s_waitcnt vmcnt(" #n ")" ::: "memory")

// Starts the copy of 16 bytes a lane, from its own offset, to 1 KB of LDS in
// lane order.
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t from, OB_LDS unsigned char *to, int offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (OB_LDS void *)to, 16, offset, 0, 0, 0);
}

// A workgroup's place: consecutive workgroups go to the 8 XCDs in turn, so
// the tiles are numbered such that each XCD (its own L2) gets a consecutive
// range: one slice of the contraction where there are several, and within it
// kGroup tiles along dY's columns times a run along X's, the shape that needs
// the fewest bytes of both (dY has two bytes an element, X one).
constexpr int kXcds = 8, kGroup = 4;
struct Where {
  int mt, nt, split;
};
__device__ __forceinline__ Where where(int m_tiles, int n_tiles, int splits) {
  const uint32_t tiles = static_cast<uint32_t>(m_tiles) * n_tiles, total = tiles * splits;
  const uint32_t id = blockIdx.x, xcd = id % kXcds, at = id / kXcds;
  const uint32_t each = total / kXcds, more = total % kXcds;
  const uint32_t lin = xcd * each + min(xcd, more) + at;
  const uint32_t split = lin / tiles, t = lin - split * tiles;
  const uint32_t band = t / (kGroup * n_tiles), in_band = t - band * kGroup * n_tiles;
  const uint32_t high = min(static_cast<uint32_t>(kGroup), m_tiles - band * kGroup);
  return Where{static_cast<int>(band * kGroup + in_band % high), static_cast<int>(in_band / high), static_cast<int>(split)};
}

template <int BM, int BN, int WM, int WN, int FMT>
__global__ __launch_bounds__(64 * WM * WN) void linear_grad_wide_kernel(const LinearArgs a, int m_tiles, int n_tiles,
                                                                       int splits, int64_t turns_each, float *part) {
  constexpr int BK = 64, NW = WM * WN, NT = 64 * NW;
  constexpr int FO = BM / WM / 16, FI = BN / WN / 16;
  constexpr int A_BYTES = BK * BM * 2, B_BYTES = BK * BN, S_BYTES = 2 * BN;
  constexpr int STAGE = A_BYTES + B_BYTES + S_BYTES;
  constexpr int JA = A_BYTES / 1024 / NW, JB = B_BYTES / 1024 / NW;   // 1 KB copies a wavefront makes each turn
  constexpr int RA = 512 / BM, RB = 1024 / BN;                        // rows of one copy
  static_assert(S_BYTES <= NT && FI % 4 == 0 && JA * NW * 1024 == A_BYTES && JB * NW * 1024 == B_BYTES, "tile shape");
  static_assert(1 + JA + JB == 7, "the waits below count a turn's loads");
  __shared__ __attribute__((aligned(1024))) unsigned char shared[3 * STAGE];
  OB_LDS unsigned char *const lds = (OB_LDS unsigned char *)shared;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const Where at = where(m_tiles, n_tiles, splits);
  const int64_t m0 = static_cast<int64_t>(at.mt) * BM, n0 = static_cast<int64_t>(at.nt) * BN;
  const int64_t turn0 = at.split * turns_each;
  const int turns = static_cast<int>(max(int64_t{0}, min(turns_each, (a.rows + BK - 1) / BK - turn0)));

  f32x4 acc[FI][FO];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int o = 0; o < FO; ++o) acc[i][o] = f32x4{0, 0, 0, 0};

  // where this lane's 16 bytes of each copy come from (the swizzle is applied
  // to the source: the copies write LDS in order)
  int from_a[JA], from_b[JB];
#pragma unroll
  for (int j = 0; j < JA; ++j) {
    const int r = (wave * JA + j) * RA + lane / (BM / 8), c = lane % (BM / 8);
    from_a[j] = static_cast<int>(r * a.lddy) * 2 + (((c >> 1) ^ swizzle_a(r)) << 5) + (c & 1) * 16;
  }
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    const int r = (wave * JB + j) * RB + lane / (BN / 16), c = lane % (BN / 16);
    from_b[j] = static_cast<int>(r * a.pitch) + ((c ^ swizzle_b<BN>(r)) << 4);
  }
  const int from_s = tid < S_BYTES ? static_cast<int>(tid / BN * a.pitch) + tid % BN : 0;
  const int to_s = tid / BN * BN + (tid % BN & 15) * (BN / 16) + (tid % BN >> 4);
  const int64_t dy_bytes = ((a.rows - 1) * a.lddy + a.out) * 2, code_bytes = a.rows * a.pitch,
                scale_bytes = act_blocks(a.rows) * a.pitch;

  // The loads of a turn; a turn past the last reads nothing and fills zeros.
  auto load_scale = [&](int turn) -> uint32_t {
    const int64_t t0 = (turn0 + turn) * BK;
    const auto r = rest(a.scales, turn < turns ? t0 / kActBlock * a.pitch + n0 : scale_bytes, scale_bytes);
    return __builtin_amdgcn_raw_buffer_load_b8(r, from_s, 0, 0);
  };
  auto copy = [&](int turn, OB_LDS unsigned char *dst) {
    const int64_t t0 = (turn0 + turn) * BK;
    const auto ra = rest(a.dy, turn < turns ? (t0 * a.lddy + m0) * 2 : (dy_bytes + 15) / 16 * 16, dy_bytes);
    const auto rb = rest(a.codes, turn < turns ? t0 * a.pitch + n0 : code_bytes, code_bytes);
#pragma unroll
    for (int j = 0; j < JA; ++j)
      copy16(ra, dst + (wave * JA + j) * 1024, from_a[j]);
#pragma unroll
    for (int j = 0; j < JB; ++j)
      copy16(rb, dst + A_BYTES + (wave * JB + j) * 1024, from_b[j]);
  };

  const int g = lane >> 4, li = lane & 15;
  const int a_row = 8 * g + (li >> 2), a_sw = (li >> 2) | (g & 1) << 2;
  const int b_row = 8 * g + (li >> 1), b_sw = swizzle_b<BN>(b_row);

  struct Step {
    uint32_t s[FI / 4];
    i32x2 c[FI];
    s16x4 y[FO][2];
  };
  auto fetch = [&](OB_LDS const unsigned char *A, int kk, Step &f) {
    OB_LDS const unsigned char *B = A + A_BYTES, *S = B + B_BYTES;
#pragma unroll
    for (int q = 0; q < FI / 4; ++q)
      f.s[q] = *(OB_LDS const uint32_t *)(S + kk * BN + li * (BN / 16) + wn * FI + 4 * q);
#pragma unroll
    for (int i = 0; i < FI; ++i)
      f.c[i] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (OB_LDS i32x2 *)(B + (kk * 32 + b_row) * BN + (((wn * FI + i) ^ b_sw) << 4) + (li & 1) * 8));
#pragma unroll
    for (int o = 0; o < FO; ++o) {
      OB_LDS const unsigned char *p = A + (kk * 32 + a_row) * (BM * 2) + (((wm * FO + o) ^ a_sw) << 5) + (li & 3) * 8;
      f.y[o][0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((OB_LDS s16x4 *)(p));
      f.y[o][1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((OB_LDS s16x4 *)(p + 4 * BM * 2));
    }
  };
  auto multiply = [&](const Step &f) {
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      const float scale = act_scale_value((f.s[i >> 2] >> (8 * (i & 3))) & 0xffu);
      const bf16x2 d[4] = {act_decode2<FMT, false>(f.c[i][0], scale), act_decode2<FMT, true>(f.c[i][0], scale),
                           act_decode2<FMT, false>(f.c[i][1], scale), act_decode2<FMT, true>(f.c[i][1], scale)};
      bf16x8 x;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = d[k >> 1][k & 1];
#pragma unroll
      for (int o = 0; o < FO; ++o) {
        const bf16x8 y = __builtin_bit_cast(bf16x8, __builtin_shufflevector(f.y[o][0], f.y[o][1], 0, 1, 2, 3, 4, 5, 6, 7));
        acc[i][o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, acc[i][o], 0, 0, 0);
      }
    }
  };

  Step f0, f1;
  uint32_t s_reg;
  // One turn on tile `cur`, tile t + 1 lying in `next`, tile t + 2 being
  // copied to `dst`: three different stages, which __restrict says, so that
  // the compiler does not hold the reads back for the copies; the waits and
  // the barrier in the middle are what orders them.
  auto turn = [&](int t, OB_LDS unsigned char *__restrict dst, OB_LDS unsigned char *__restrict cur,
                  OB_LDS unsigned char *__restrict next) __attribute__((always_inline)) {
    fetch(cur, 1, f1);
    if (S_BYTES == NT || tid < S_BYTES) next[A_BYTES + B_BYTES + to_s] = static_cast<unsigned char>(s_reg);
    s_reg = load_scale(t + 2);
    copy(t + 2, dst);
    __builtin_amdgcn_sched_barrier(0);
    multiply(f0);
    __builtin_amdgcn_sched_barrier(0);
    // tile t + 1 has landed once only this turn's 7 loads are out; this
    // wavefront's reads of tile t are back
    asm volatile("s_waitcnt vmcnt(7) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    fetch(next, 0, f0);
    __builtin_amdgcn_sched_barrier(0);
    multiply(f1);
    __builtin_amdgcn_sched_barrier(0);
  };

  if (turns > 0) {
    const uint32_t s0 = load_scale(0);
    copy(0, lds);
    s_reg = load_scale(1);
    copy(1, lds + STAGE);
    if (S_BYTES == NT || tid < S_BYTES) lds[A_BYTES + B_BYTES + to_s] = static_cast<unsigned char>(s0);
    asm volatile("s_waitcnt vmcnt(7) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    fetch(lds, 0, f0);
    OB_LDS unsigned char *cur = lds, *next = lds + STAGE, *dst = lds + 2 * STAGE;
    for (int t = 0; t < turns; ++t) {
      turn(t, dst, cur, next);
      OB_LDS unsigned char *const was = cur;
      cur = next;
      next = dst;
      dst = was;
    }
    OB_WAIT_VM(0);   // no copy may land after the workgroup has ended
  }
  store_tile<BM, BN, WM, WN, FO, FI>(a, acc, m0, n0, wm, wn, part ? part + at.split * a.out * a.in : nullptr);
}

// Column sums of dY over slices of rows: lane per column, the four wavefronts
// take every fourth row of the slice, added in order.
template <typename T>
__global__ __launch_bounds__(256) void bias_kernel(const LinearArgs a, float *part, int64_t rows_each) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const int64_t r0 = blockIdx.y * rows_each, r1 = min(a.rows, r0 + rows_each);
  float sum = 0.0f;
  if (col < a.out) {
#pragma unroll 8
    for (int64_t r = r0 + wave; r < r1; r += 4) {
      const T v = static_cast<const T *>(a.dy)[r * a.lddy + col];
      if constexpr (sizeof(T) == 4) sum += v;
      else sum += __uint_as_float(static_cast<uint32_t>(v) << 16);
    }
  }
  __shared__ float s[4][64];
  s[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && col < a.out)
    part[blockIdx.y * a.out + col] = ((s[0][lane] + s[1][lane]) + s[2][lane]) + s[3][lane];
}

// out[e] = (accumulate ? out[e] : 0) + sum of the parts in order.
template <typename G>
__global__ __launch_bounds__(kBlock) void join_parts_kernel(const float *part, int parts, int64_t n, void *out,
                                                            bool accumulate) {
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x) * 4;
  if (first >= n) return;
  G *p = static_cast<G *>(out) + first;
  const bool quad = n % 4 == 0;
  f32x4 v = {0, 0, 0, 0};
  for (int s = 0; s < parts; ++s) {
    const float *q = part + s * n + first;
    if (quad) {
      v += *reinterpret_cast<const f32x4 *>(q);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (first + k < n) v[k] += q[k];
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (first + k < n) {
      if constexpr (sizeof(G) == 4) p[k] = accumulate ? p[k] + v[k] : v[k];
      else
        p[k] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(
                   accumulate ? __uint_as_float(static_cast<uint32_t>(p[k]) << 16) + v[k] : v[k]));
    }
  }
}

constexpr int kBiasRows = 512;

struct Plan {
  int bm, bn, bk;
  int m_tiles, n_tiles;
  int64_t turns_each;
  int splits;                // parts of the contraction; > 1: joined from the workspace
  int bias_slices;
  size_t weight_bytes, bias_bytes;
};

Plan plan_of(int64_t rows, int64_t out, int64_t in, bool dy_bf16, bool bias) {
  Plan p{};
  p.bm = p.bn = dy_bf16 && ((out + 255) / 256) * ((in + 255) / 256) >= 128 ? 256 : 128;
  p.bk = dy_bf16 ? 64 : 32;
  p.m_tiles = static_cast<int>((out + p.bm - 1) / p.bm);
  p.n_tiles = static_cast<int>((in + p.bn - 1) / p.bn);
  const int64_t turns = (rows + p.bk - 1) / p.bk;
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  // enough workgroups for the 256 CUs, at least 8 turns each
  int64_t splits = tiles >= 256 ? 1 : (512 + tiles - 1) / tiles;
  splits = splits > turns / 8 ? turns / 8 : splits;
  if (splits < 1) splits = 1;
  p.turns_each = turns ? (turns + splits - 1) / splits : 0;
  p.splits = static_cast<int>(turns ? (turns + p.turns_each - 1) / p.turns_each : 1);
  p.bias_slices = bias ? static_cast<int>(rows ? (rows + kBiasRows - 1) / kBiasRows : 1) : 0;
  p.weight_bytes = p.splits > 1 ? (static_cast<size_t>(p.splits) * out * in * 4 + 255) / 256 * 256 : 0;
  p.bias_bytes = static_cast<size_t>(p.bias_slices) * out * 4;
  return p;
}

Plan plan_of(const LinearArgs &a) { return plan_of(a.rows, a.out, a.in, a.dy_bf16, a.db != nullptr); }

template <int BM, int BN, int BK, int WM, int WN, int PARTS>
void linear_one(const LinearArgs &a, const Plan &p, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.m_tiles) * p.n_tiles, p.splits);
  float *part = p.splits > 1 ? static_cast<float *>(a.work) : nullptr;
  const int64_t size = PARTS == 1 ? 2 : 4;
  const bool vec = reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 && a.lddy * size % 16 == 0 &&
                   (a.lddy * BK + a.out) * size < 0x7fffffff;
  if (a.fmt == kE4M3) {
    if (vec) linear_grad_kernel<BM, BN, BK, WM, WN, PARTS, kE4M3, true><<<grid, 64 * WM * WN, 0, s>>>(a, p.m_tiles, p.n_tiles, p.turns_each, part);
    else linear_grad_kernel<BM, BN, BK, WM, WN, PARTS, kE4M3, false><<<grid, 64 * WM * WN, 0, s>>>(a, p.m_tiles, p.n_tiles, p.turns_each, part);
  } else {
    if (vec) linear_grad_kernel<BM, BN, BK, WM, WN, PARTS, kInt8, true><<<grid, 64 * WM * WN, 0, s>>>(a, p.m_tiles, p.n_tiles, p.turns_each, part);
    else linear_grad_kernel<BM, BN, BK, WM, WN, PARTS, kInt8, false><<<grid, 64 * WM * WN, 0, s>>>(a, p.m_tiles, p.n_tiles, p.turns_each, part);
  }
}

template <int BM, int BN, int WM, int WN>
void linear_wide(const LinearArgs &a, const Plan &p, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.m_tiles) * p.n_tiles * p.splits);
  float *part = p.splits > 1 ? static_cast<float *>(a.work) : nullptr;
  if (a.fmt == kE4M3)
    linear_grad_wide_kernel<BM, BN, WM, WN, kE4M3><<<grid, 64 * WM * WN, 0, s>>>(a, p.m_tiles, p.n_tiles, p.splits, p.turns_each, part);
  else
    linear_grad_wide_kernel<BM, BN, WM, WN, kInt8><<<grid, 64 * WM * WN, 0, s>>>(a, p.m_tiles, p.n_tiles, p.splits, p.turns_each, part);
}

}  // namespace

bool linear_fits(int64_t rows, int64_t out, int64_t in) {
  // a turn's codes lie within 2 GB; tiles and row slices within the grid's limits
  return in <= (int64_t{1} << 24) && out <= (int64_t{1} << 31) && rows <= (int64_t{1} << 24) &&
         ((out + 127) / 128) * ((in + 127) / 128) <= kMaxGrid;
}

size_t linear_work_bytes(int64_t rows, int64_t out, int64_t in, bool dy_bf16, bool bias) {
  const Plan p = plan_of(rows, out, in, dy_bf16, bias);
  return p.weight_bytes + p.bias_bytes;
}

void launch_linear_grad(const LinearArgs &a, hipStream_t s) {
  const Plan p = plan_of(a);
  if (a.dy_bf16 && p.bm == 256) linear_wide<256, 256, 4, 2>(a, p, s);
  else if (a.dy_bf16) linear_one<128, 128, 64, 2, 2, 1>(a, p, s);
  else linear_one<128, 128, 32, 2, 2, 3>(a, p, s);
  if (a.db) {
    float *part = reinterpret_cast<float *>(static_cast<char *>(a.work) + p.weight_bytes);
    const dim3 grid(static_cast<unsigned>((a.out + 63) / 64), p.bias_slices);
    if (a.dy_bf16) bias_kernel<uint16_t><<<grid, 256, 0, s>>>(a, part, kBiasRows);
    else bias_kernel<float><<<grid, 256, 0, s>>>(a, part, kBiasRows);
  }
}

bool linear_needs_join(const LinearArgs &a) { return a.db != nullptr || plan_of(a).splits > 1; }

void launch_linear_join(const LinearArgs &a, hipStream_t s) {
  const Plan p = plan_of(a);
  const auto join = [&](const float *part, int parts, int64_t n, void *out) {
    const dim3 grid(static_cast<unsigned>((n + 4 * kBlock - 1) / (4 * kBlock)));
    if (a.grad_bf16) join_parts_kernel<uint16_t><<<grid, kBlock, 0, s>>>(part, parts, n, out, a.accumulate);
    else join_parts_kernel<float><<<grid, kBlock, 0, s>>>(part, parts, n, out, a.accumulate);
  };
  if (p.splits > 1) join(static_cast<const float *>(a.work), p.splits, a.out * a.in, a.dw);
  if (a.db)
    join(reinterpret_cast<const float *>(static_cast<const char *>(a.work) + p.weight_bytes), p.bias_slices, a.out, a.db);
}

}  // namespace ob
