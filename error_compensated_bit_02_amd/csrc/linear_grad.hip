// Weight and bias gradient of a linear layer from an 8-bit checkpoint of its
// input (gfx950):
//   dW[o][i] = sum over t of dY[t][o] * X[t][i],   db[o] = sum over t of dY[t][o]
// with X the checkpoint's values.  The result goes straight into one worker's
// gradient row of the tensor list.
//
// The contraction runs on the bf16 matrix units with fp32 accumulators.  X is
// exact in bf16 (activation.h), so with bf16 dY the products are exact.  An
// fp32 dY is cut into three bf16 parts of 8 significant bits each, which add
// up to it exactly but for bits below bf16's last, 2^-133; three products per
// element keep fp32 accuracy at a third of the bf16 rate.
//
// Both operands lie with the contraction index t slowest ([t][o] and [t][i]),
// and a matrix instruction wants 8 consecutive t per lane: the tiles go to LDS
// as they are and come back transposed (ds_read_b64_tr_b16 for dY,
// ds_read_b64_tr_b8 for the codes).  The codes stay bytes in LDS and are
// converted after the read, one scale per lane and 32 tokens.  X is the
// instruction's first operand, so a lane's four results are four consecutive
// i of one weight row, stored as one vector.
//
// Precision.  Sums are fp32 throughout, the parts of a split contraction too;
// the only rounding to fewer bits is the one to the gradient's type at the end.
//
// Measured on MI355X (a call, bias included).  8192 x 2048 over 16384 tokens, bf16
// dY: 400 us with e4m3 (396 to 430 as the card's clock goes, 1280-1390 TFLOP/s; the
// library's bf16 product of that shape, X in bf16 and no bias, 457 us), 470 us with
// int8, whose conversion takes five vector instructions for two elements instead
// of one.  With constant inputs it takes 340 us: the card lowers its clock under
// load.  1024 x 1024 over 4096 tokens 30 us, in fp32 50: 256 (512) workgroups of 16
// turns.  A lone tile's turn takes 0.82 us where its products need 0.21: one
// wavefront a SIMD has nobody to fill its waits (the matrix units are busy 12% of
// the kernel's cycles, 64% in the large case); start, end, the split's parts and
// the join are the rest.  1000 x 2048 over 777 in fp32 35 us, 4096 x 4096 over 8192
// 807.
#include "internal.h"
#include "activation.h"
#include "tiles.h"

#include <algorithm>

#pragma clang fp contract(off)

namespace ob {
namespace {

// The codes' rows likewise, in units of 16 bytes.
template <int BN>
__device__ __forceinline__ int swizzle_b(int r) {
  return BN >= 256 ? ((r & 7) | ((r >> 3) & 1) << 3) : (r & 7);
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


// Sum of a lane's eight values of a dY fragment.
__device__ __forceinline__ float fragment_sum(s16x4 lo, s16x4 hi) {
  const i32x2 a = __builtin_bit_cast(i32x2, lo), b = __builtin_bit_cast(i32x2, hi);
  const auto even = [](int w) { return __int_as_float(w << 16); };
  const auto odd = [](int w) { return __int_as_float(w & static_cast<int>(0xffff0000u)); };
  return ((even(a[0]) + odd(a[0])) + (even(a[1]) + odd(a[1]))) + ((even(b[0]) + odd(b[0])) + (even(b[1]) + odd(b[1])));
}

// This workgroup's part of the bias gradient: one row of `part`.
template <int FO, int WN>
__device__ __forceinline__ void store_columns(const LinearArgs &a, float (&sum)[FO / WN], int64_t m0, int wm, int wn, float *part) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 0; o < FO / WN; ++o) {
    float v = sum[o];
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    const int64_t row = m0 + (wm * FO + wn * (FO / WN) + o) * 16 + lane;
    if (lane < 16 && row < a.out) part[row] = v;
  }
}

// Drops the first `s` (0..7) of eight elements, N 32-bit words of them; zeros move in.
template <int N>
__device__ __forceinline__ void drop_front(uint32_t (&w)[N], int s) {
  if (s & 4) {
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = k + N / 2 < N ? w[k + N / 2] : 0;
  }
  if (s & 2) {
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = k + N / 4 < N ? w[k + N / 4] : 0;
  }
  if (s & 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t up = k + 1 < N ? w[k + 1] : 0;
      w[k] = N == 8 ? up : (w[k] >> 16 | up << 16);
    }
  }
}

// One workgroup's tile of dW over one slice of the contraction.
//
// BM x BN is the tile, WM x WN its wavefronts; a turn is BK tokens.  T is dY's
// element (uint16_t: bf16; float: cut into three parts).  COPY: dY goes
// straight from memory to LDS, 16 bytes a lane (bf16 whose rows start on 16
// bytes); otherwise through registers, which costs them one turn of delay.
// The codes always go straight to LDS.
//
// Stages.  At turn t the products run on tile t, tile t + 1 has arrived or is
// arriving, and the copies of tile t + 2 start.  One barrier a turn: behind
// it tile t + 1 is in LDS and nobody reads tile t any more.  Within a turn
// every step's operands are read one step ahead of its products, so the
// matrix unit has work while LDS answers.
template <int BM, int BN, int BK, int WM, int WN, typename T, int FMT, bool COPY>
__global__ __launch_bounds__(64 * WM * WN, 2) void linear_grad_kernel(const LinearArgs a, const Split sp, float *part, float *bias_part) {
  constexpr int PARTS = sizeof(T) == 2 ? 1 : 3;
  constexpr int NW = WM * WN, NT = 64 * NW, KK = BK / 32;
  constexpr int FO = BM / WM / 16, FI = BN / WN / 16;                 // fragments of a wavefront
  constexpr int A_BYTES = BK * BM * 2, B_BYTES = BK * BN, S_BYTES = KK * BN;
  constexpr int A_STAGE = PARTS * A_BYTES, B_STAGE = B_BYTES + (S_BYTES + 255) / 256 * 256;
  constexpr int STAGES = 3, A_STAGES = COPY ? STAGES : 2;         // through registers dY arrives a turn later
  constexpr int JA = COPY ? A_BYTES / 1024 / NW : BK * BM / 8 / NT;   // dY: copies, or 8-element loads
  constexpr int JB = B_BYTES / 1024 / NW;
  constexpr int RA = 512 / BM, RB = 1024 / BN;                        // rows of one copy
  static_assert(!COPY || PARTS == 1, "fp32 goes through registers");
  static_assert(FI % 4 == 0 && FO % WN == 0 && JB * NW * 1024 == B_BYTES && JA >= 1, "tile shape");
  static_assert(!COPY || JA * NW * 1024 == A_BYTES, "tile shape");
  __shared__ __attribute__((aligned(1024))) unsigned char shared[A_STAGES * A_STAGE + STAGES * B_STAGE];
  OB_LDS unsigned char *const lds = (OB_LDS unsigned char *)shared;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const Where at = where(sp);
  const int64_t m0 = static_cast<int64_t>(at.mt) * BM, n0 = static_cast<int64_t>(at.nt) * BN;
  const int64_t turn0 = at.split * sp.turns_each;
  const int turns = static_cast<int>(max(int64_t{0}, min(sp.turns_each, (a.rows + BK - 1) / BK - turn0)));

  f32x4 acc[FI][FO];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int o = 0; o < FO; ++o) acc[i][o] = f32x4{0, 0, 0, 0};
  float columns[FO / WN];
#pragma unroll
  for (int o = 0; o < FO / WN; ++o) columns[o] = 0.0f;

  // Where this lane's 16 bytes of each copy come from: the copies write LDS
  // in lane order, so the swizzle is applied to the source.
  int from_a[COPY ? JA : 1], from_b[JB];
  if constexpr (COPY) {
#pragma unroll
    for (int j = 0; j < JA; ++j) {
      const int r = (wave * JA + j) * RA + lane / (BM / 8), c = lane % (BM / 8);
      from_a[j] = static_cast<int>(r * a.lddy) * 2 + (((c >> 1) ^ swizzle_a(r)) << 5) + (c & 1) * 16;
    }
  }
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    const int r = (wave * JB + j) * RB + lane / (BN / 16), c = lane % (BN / 16);
    from_b[j] = static_cast<int>(r * a.pitch) + ((c ^ swizzle_b<BN>(r)) << 4);
  }
  // Scales, 256 bytes a copy: every wavefront makes one, several the same.
  constexpr int SC = (S_BYTES + 255) / 256;
  const int to_s = wave % SC * 256, from_s = (to_s + lane * 4) / BN * static_cast<int>(a.pitch) + (to_s + lane * 4) % BN;
  // Where the next turn to be started reads, and how many rows it has: none
  // past the last turn.
  const int64_t row0 = turn0 * BK;
  const char *dy_from = static_cast<const char *>(a.dy) + (row0 * a.lddy + m0) * static_cast<int>(sizeof(T));
  const uint8_t *codes_from = a.codes + row0 * a.pitch + n0, *scales_from = a.scales + row0 / kActBlock * a.pitch + n0;
  const int pitch = static_cast<int>(a.pitch);
  int rows_left = static_cast<int>(min(a.rows - row0, static_cast<int64_t>(turns) * BK));

  // What passes through registers, a turn at a time.
  constexpr int CA = BM / 8, RT = NT / CA;             // chunks of a dY row, rows of one step
  const int ca = tid % CA, ra = tid / CA;
  uint32_t dy_reg[COPY ? 1 : JA][2 * sizeof(T)];

  // dY through registers: a lane's eight elements are read wherever they lie,
  // those past a row's end (dropped later) being the next row's.  Only at the
  // very end of the matrix (of kFewRows elements at least) the read is moved
  // back inside it, and settle() drops what came in front.
  const int64_t dy_count = (a.rows - 1) * a.lddy + a.out;
  const auto dy_at = [&](int64_t row) __attribute__((always_inline)) {
    const int64_t m = m0 + ca * 8;
    return row * a.lddy + (m < a.out ? m : 0);
  };

  // Starts the loads of the next turn.
  auto start = [&](int turn, OB_LDS unsigned char *a_dst, OB_LDS unsigned char *b_dst) __attribute__((always_inline)) {
    // its rows, and all ones or zeros by whether it has any
    const int n = max(0, min(rows_left, BK)), any = -n >> 31;
    rows_left -= BK;
    const auto rs = buffer(scales_from, ((n + kActBlock - 1) / kActBlock * pitch - static_cast<int>(n0)) & any);
    copy4(rs, b_dst + B_BYTES + to_s, from_s);
    scales_from += KK * pitch;
    if constexpr (COPY) {
      const int ld = static_cast<int>(a.lddy);
      const auto rd = buffer(dy_from, ((n - 1) * ld + static_cast<int>(a.out - m0)) * 2 & any);
#pragma unroll
      for (int j = 0; j < JA; ++j) copy16(rd, a_dst + (wave * JA + j) * 1024, from_a[j]);
      dy_from += BK * a.lddy * 2;
    } else {
#pragma unroll
      for (int j = 0; j < JA; ++j) {
        const int64_t e = min(dy_at(n > 0 ? row0 + turn * BK + ra + RT * j : 0), dy_count - 8);
        __builtin_memcpy(dy_reg[j], static_cast<const T *>(a.dy) + e, 8 * sizeof(T));
      }
    }
    const auto rc = buffer(codes_from, (n * pitch - static_cast<int>(n0)) & any);
#pragma unroll
    for (int j = 0; j < JB; ++j) copy16(rc, b_dst + (wave * JB + j) * 1024, from_b[j]);
    codes_from += BK * pitch;
  };
  // Puts what came through registers for a turn into its tile.
  auto settle = [&](int turn, OB_LDS unsigned char *a_to) __attribute__((always_inline)) {
    if constexpr (!COPY) {
      const int64_t t0 = row0 + turn * BK;
      if (t0 + BK + 8 > a.rows) {          // the rows may end here
#pragma unroll
        for (int j = 0; j < JA; ++j) {
          const int64_t row = t0 + ra + RT * j, e = dy_at(row);
          if (row >= a.rows) {
#pragma unroll
            for (uint32_t &w : dy_reg[j]) w = 0;
          } else if (e > dy_count - 8) {
            drop_front(dy_reg[j], static_cast<int>(min(int64_t{7}, e - (dy_count - 8))));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < JA; ++j) {
        const int r = ra + RT * j;
        OB_LDS unsigned char *p = a_to + r * (BM * 2) + (((ca >> 1) ^ swizzle_a(r)) << 5) + (ca & 1) * 16;
        if constexpr (PARTS == 1) {
          *(OB_LDS i32x4 *)p = i32x4{static_cast<int>(dy_reg[j][0]), static_cast<int>(dy_reg[j][1]),
                                     static_cast<int>(dy_reg[j][2]), static_cast<int>(dy_reg[j][3])};
        } else {
          i32x4 w[3];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h[2], m[2], l[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) split3(__uint_as_float(dy_reg[j][2 * k + e]), h[e], m[e], l[e]);
            w[0][k] = static_cast<int>(h[0] | h[1] << 16);
            w[1][k] = static_cast<int>(m[0] | m[1] << 16);
            w[2][k] = static_cast<int>(l[0] | l[1] << 16);
          }
#pragma unroll
          for (int q = 0; q < 3; ++q) *(OB_LDS i32x4 *)(p + q * A_BYTES) = w[q];
        }
      }
    }
  };
  // The loads of turn t + 1 are done once only those of the turns after it are
  // out (an access of 16 bytes is one load at least).
  constexpr int kLoads = 1 + JA * (PARTS == 1 ? 1 : 2) + JB, kOut = (STAGES - 2) * kLoads;
  auto arrived = [&]() __attribute__((always_inline)) {
    wait_loads<kOut>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  const int g = lane >> 4, li = lane & 15;
  const int a_row = 8 * g + (li >> 2), a_sw = (li >> 2) | (g & 1) << 2;
  const int b_row = 8 * g + (li >> 1), b_sw = swizzle_b<BN>(b_row);

  // Operands of one 32-token step as they come from LDS: the codes with their
  // scales, and dY (one of its parts).
  struct Codes {
    uint32_t s[FI];
    i32x2 c[FI];
  };
  struct Dy {
    s16x4 y[FO][2];
  };
  auto fetch_codes = [&](OB_LDS const unsigned char *B, int kk, Codes &f) __attribute__((always_inline)) {
    OB_LDS const unsigned char *S = B + B_BYTES;
#pragma unroll
    for (int i = 0; i < FI; ++i) f.s[i] = S[kk * BN + (wn * FI + i) * 16 + li];
#pragma unroll
    for (int i = 0; i < FI; ++i)
      f.c[i] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (OB_LDS i32x2 *)(B + (kk * 32 + b_row) * BN + (((wn * FI + i) ^ b_sw) << 4) + (li & 1) * 8));
  };
  auto fetch_dy = [&](OB_LDS const unsigned char *A, int kk, Dy &f) __attribute__((always_inline)) {
#pragma unroll
    for (int o = 0; o < FO; ++o) {
      OB_LDS const unsigned char *p = A + (kk * 32 + a_row) * (BM * 2) + (((wm * FO + o) ^ a_sw) << 5) + (li & 3) * 8;
      f.y[o][0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((OB_LDS s16x4 *)(p));
      f.y[o][1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((OB_LDS s16x4 *)(p + 4 * BM * 2));
    }
  };
  auto decode = [&](const Codes &f, int i) __attribute__((always_inline)) -> bf16x8 {
    const float scale = act_scale_value(f.s[i]);
    const bf16x2 d[4] = {act_decode2<FMT, false>(f.c[i][0], scale), act_decode2<FMT, true>(f.c[i][0], scale),
                         act_decode2<FMT, false>(f.c[i][1], scale), act_decode2<FMT, true>(f.c[i][1], scale)};
    bf16x8 x;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = d[k >> 1][k & 1];
    return x;
  };
  auto multiply = [&](const bf16x8 &x, const Dy &f, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int o = 0; o < FO; ++o) {
      const bf16x8 y = __builtin_bit_cast(bf16x8, __builtin_shufflevector(f.y[o][0], f.y[o][1], 0, 1, 2, 3, 4, 5, 6, 7));
      acc[i][o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, acc[i][o], 0, 0, 0);
    }
  };
  // Column sums of a step's dY: the WN wavefronts that share a fragment divide
  // them.
  auto add_columns = [&](const Dy &f) __attribute__((always_inline)) {
#pragma unroll
    for (int o = 0; o < FO; ++o)
      if (wn == o / (FO / WN)) columns[o % (FO / WN)] += fragment_sum(f.y[o][0], f.y[o][1]);
  };
  int sum_in = at.nt;              // turns until this workgroup's next share of the column sums

  // Spreads the reads between the products: the wavefronts of a SIMD come out
  // of the barrier together, and a run of reads would fill the LDS queue while
  // the matrix unit stands still.
  auto interleave = [&]() __attribute__((always_inline)) {
    constexpr int kReads = 2 * FI + 2 * FO;
#pragma unroll
    for (int k = 0; k < kReads; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one product
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one read
    }
  };

  // One turn.  The stages differ, which __restrict says: the compiler would
  // otherwise hold every read back until all copies have landed.  The
  // scheduling fences keep the reads ahead of the products before them.
  // bf16: two steps, the first one's operands in (c, p) and the next turn's
  // left there again.
  auto turn_bf16 = [&](int t, Codes &c, Codes &d, Dy &p, Dy &q, OB_LDS unsigned char *__restrict a_dst,
                       OB_LDS unsigned char *__restrict a_cur, OB_LDS unsigned char *__restrict a_next,
                       OB_LDS unsigned char *__restrict b_dst, OB_LDS unsigned char *__restrict b_cur,
                       OB_LDS unsigned char *__restrict b_next) __attribute__((always_inline)) {
    const bool sums = bias_part != nullptr && sum_in == 0;
    sum_in = sum_in == 0 ? sp.n_tiles - 1 : sum_in - 1;
    settle(t + 1, a_next);
    start(t + STAGES - 1, a_dst, b_dst);
    if (sums) add_columns(p);
    __builtin_amdgcn_sched_barrier(0);
    fetch_codes(b_cur, 1, d);
    fetch_dy(a_cur, 1, q);
#pragma unroll
    for (int i = 0; i < FI; ++i) multiply(decode(c, i), p, i);
    interleave();
    __builtin_amdgcn_sched_barrier(0);
    arrived();
    if (sums) add_columns(q);
    __builtin_amdgcn_sched_barrier(0);
    fetch_codes(b_next, 0, c);
    fetch_dy(a_next, 0, p);
#pragma unroll
    for (int i = 0; i < FI; ++i) multiply(decode(d, i), q, i);
    interleave();
    __builtin_amdgcn_sched_barrier(0);
  };
  // fp32: one step in three parts, the first one's operands in (c, p), the
  // next turn's left in (c, q).
  auto turn_f32 = [&](int t, Codes &c, Dy &p, Dy &q, OB_LDS unsigned char *__restrict a_cur,
                      OB_LDS unsigned char *__restrict a_next, OB_LDS unsigned char *__restrict b_dst,
                      OB_LDS unsigned char *__restrict b_next) __attribute__((always_inline)) {
    const bool sums = bias_part != nullptr && sum_in == 0;
    sum_in = sum_in == 0 ? sp.n_tiles - 1 : sum_in - 1;
    bf16x8 x[FI];
#pragma unroll
    for (int i = 0; i < FI; ++i) x[i] = decode(c, i);
    fetch_dy(a_cur + A_BYTES, 0, q);
    settle(t + 1, a_next);
    start(t + STAGES - 1, nullptr, b_dst);
    __builtin_amdgcn_sched_barrier(0);
    if (sums) add_columns(p);
#pragma unroll
    for (int i = 0; i < FI; ++i) multiply(x[i], p, i);
    fetch_dy(a_cur + 2 * A_BYTES, 0, p);
    __builtin_amdgcn_sched_barrier(0);
    if (sums) add_columns(q);
#pragma unroll
    for (int i = 0; i < FI; ++i) multiply(x[i], q, i);
    __builtin_amdgcn_sched_barrier(0);
    arrived();
    fetch_codes(b_next, 0, c);
    fetch_dy(a_next, 0, q);
    __builtin_amdgcn_sched_barrier(0);
    if (sums) add_columns(p);
#pragma unroll
    for (int i = 0; i < FI; ++i) multiply(x[i], p, i);
    __builtin_amdgcn_sched_barrier(0);
  };

  if (turns > 0) {
    // stages by turn: cur, next and the one that the copies started now go to
    int a_at = 0, b_at = 0;
    const auto a_stage = [&](int k) __attribute__((always_inline)) {
      const int n = a_at + k;
      return lds + (n >= A_STAGES ? n - A_STAGES : n) * A_STAGE;
    };
    const auto b_stage = [&](int k) __attribute__((always_inline)) {
      const int n = b_at + k;
      return lds + A_STAGES * A_STAGE + (n >= STAGES ? n - STAGES : n) * B_STAGE;
    };
    const auto rotate = [&]() __attribute__((always_inline)) {
      a_at = a_at + 1 == A_STAGES ? 0 : a_at + 1;
      b_at = b_at + 1 == STAGES ? 0 : b_at + 1;
    };
    Codes c0;
    Dy y0, y1;
    start(0, a_stage(0), b_stage(0));
    settle(0, a_stage(0));
#pragma unroll
    for (int k = 1; k < STAGES - 1; ++k) start(k, a_stage(k), b_stage(k));
    arrived();
    fetch_codes(b_stage(0), 0, c0);
    fetch_dy(a_stage(0), 0, y0);
    if constexpr (PARTS == 1) {
      static_assert(PARTS != 1 || KK == 2, "two steps a turn");
      Codes c1;
      for (int t = 0; t < turns; ++t) {
        turn_bf16(t, c0, c1, y0, y1, a_stage(A_STAGES - 1), a_stage(0), a_stage(1), b_stage(STAGES - 1), b_stage(0), b_stage(1));
        rotate();
      }
    } else {
      static_assert(PARTS == 1 || KK == 1, "one step a turn");
      for (int t = 0; t < turns; t += 2) {
        turn_f32(t, c0, y0, y1, a_stage(0), a_stage(1), b_stage(STAGES - 1), b_stage(1));
        rotate();
        if (t + 1 >= turns) break;
        turn_f32(t + 1, c0, y1, y0, a_stage(0), a_stage(1), b_stage(STAGES - 1), b_stage(1));
        rotate();
      }
    }
    wait_loads<0>();   // no copy may land after the workgroup has ended
  }
  store_tile<BM, BN, WM, WN, FO, FI>(a, acc, m0, n0, wm, wn, part ? part + at.split * a.out * a.in : nullptr);
  if (bias_part) store_columns<FO, WN>(a, columns, m0, wm, wn, bias_part + (at.split * sp.n_tiles + at.nt) * a.out);
}

// A few rows: an outer product or little more, bound by writing dW.  A thread
// holds four columns of one weight row; the first one of a row its bias too.
constexpr int kFewRows = 8;      // fewer than this
template <typename T, typename G, int FMT>
__global__ __launch_bounds__(kBlock) void linear_grad_few_kernel(const LinearArgs a, uint32_t quads) {
  const uint32_t id = blockIdx.x * kBlock + threadIdx.x;
  const uint32_t o = id / quads, i = (id - o * quads) * 4;
  if (o >= a.out) return;
  uint32_t s = 0, c[kFewRows - 1];
  float y[kFewRows - 1];
  if (a.rows > 0) s = *reinterpret_cast<const uint32_t *>(a.scales + i);
#pragma unroll
  for (int r = 0; r < kFewRows - 1; ++r) {
    c[r] = 0;
    y[r] = 0.0f;
    if (r < a.rows) {
      c[r] = *reinterpret_cast<const uint32_t *>(a.codes + r * a.pitch + i);
      const T v = static_cast<const T *>(a.dy)[r * a.lddy + o];
      if constexpr (sizeof(T) == 4) y[r] = v;
      else y[r] = __uint_as_float(static_cast<uint32_t>(v) << 16);
    }
  }
  float w[4] = {0.0f, 0.0f, 0.0f, 0.0f}, b = 0.0f;
#pragma unroll
  for (int r = 0; r < kFewRows - 1; ++r) {
    if (r < a.rows) {
      const bf16x2 lo = act_decode2<FMT, false>(c[r], 1.0f), hi = act_decode2<FMT, true>(c[r], 1.0f);
      const float x[4] = {static_cast<float>(lo[0]), static_cast<float>(lo[1]), static_cast<float>(hi[0]), static_cast<float>(hi[1])};
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = __builtin_fmaf(y[r], x[k] * act_scale_value((s >> (8 * k)) & 0xffu), w[k]);
      b += y[r];
    }
  }
  const auto put = [&](G *p, float v) {
    if constexpr (sizeof(G) == 4) *p = a.accumulate ? *p + v : v;
    else *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(a.accumulate ? __uint_as_float(static_cast<uint32_t>(*p) << 16) + v : v));
  };
  G *p = static_cast<G *>(a.dw) + static_cast<int64_t>(o) * a.in + i;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (i + k < a.in) put(p + k, w[k]);
  if (a.db && i == 0) put(static_cast<G *>(a.db) + o, b);
}

// out[e] = (accumulate ? out[e] : 0) + sum of its parts in order, for the
// weight (first `weight_blocks` workgroups) and the bias.
template <typename G>
__device__ __forceinline__ void join_parts(const float *part, int64_t parts, int64_t n, G *out, bool accumulate, int64_t first) {
  if (first >= n) return;
  G *p = out + first;
  f32x4 v = {0, 0, 0, 0};
  if (n % 4 == 0) {
#pragma unroll 4
    for (int64_t s = 0; s < parts; ++s) v += *reinterpret_cast<const f32x4 *>(part + s * n + first);
  } else {
    for (int64_t s = 0; s < parts; ++s) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (first + k < n) v[k] += part[s * n + first + k];
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

template <typename G>
__global__ __launch_bounds__(kBlock) void join_kernel(const LinearArgs a, const float *part, int64_t parts, int64_t weight_blocks,
                                                      const float *bias_part, int64_t bias_parts) {
  const int64_t b = blockIdx.x;
  if (b < weight_blocks)
    join_parts<G>(part, parts, a.out * a.in, static_cast<G *>(a.dw), a.accumulate, (b * kBlock + threadIdx.x) * 4);
  else
    join_parts<G>(bias_part, bias_parts, a.out, static_cast<G *>(a.db), a.accumulate, ((b - weight_blocks) * kBlock + threadIdx.x) * 4);
}

struct Plan {
  int tile;                  // 256 or 128: both sides of the tile
  Split sp;
  size_t weight_bytes, bias_bytes;
};

// Tile and number of slices with the least estimated time, in microseconds.
// A launch runs in rounds of as many workgroups as the 256 CUs hold: one of
// the large tile each, two of the small one.  Measured on MI355X (e4m3, bf16
// dY): a 64-token turn of the large tile 1.55 us, of one small tile on a CU
// 0.82, of two together 1.07; a workgroup's start and end 11 and 5 us; a slice
// costs the writing and reading of its fp32 part at about 3 TB/s, and the
// join.  Writing dW, which every plan does, is left out.  16384 x 2048 x 2048:
// large tile in 4 slices 126 us, small in 2 146 us; 4096 x 4096 x 1024: 52.3
// against 51.9; 16384 x 8192 x 2048: large tile whole 411 us (in 2 slices 465),
// small 549.  Where dY is not copied (or fp32) only the small tile is built: the
// large one's registers would not hold a turn of dY as well (it measured 236-277
// us against 192 at 16384 x 2048 x 2048).
// The constants are those of e4m3 with bf16 dY copied to LDS.  int8, fp32 dY and dY
// through registers are planned with the same ones, which rank slices, but are
// below their times: estimated and measured 408 and 470 us for int8 16384 x 8192 x
// 2048, 155 and 192 for dY through registers at 16384 x 2048 x 2048, 553 and 807
// for fp32 8192 x 4096 x 4096, 35 and 50 for fp32 4096 x 1024 x 1024.
Plan plan_of(int64_t rows, int64_t out, int64_t in, bool dy_bf16, bool copies, bool bias) {
  Plan p{};
  if (rows < kFewRows) return p;
  const int64_t bk = dy_bf16 ? 64 : 32, turns = (rows + bk - 1) / bk;
  const double join = 2.0, part = static_cast<double>(out) * in * 4 / 3e6;
  double best = 0.0;
  for (const int tile : {256, 128}) {
    if (tile == 256 && !copies) continue;
    const int64_t m = (out + tile - 1) / tile, n = (in + tile - 1) / tile;
    for (int64_t want = 1; want <= std::min<int64_t>(turns, 64); ++want) {
      const int64_t each = (turns + want - 1) / want, splits = (turns + each - 1) / each, groups = m * n * splits;
      if (splits != want || groups > kMaxGrid / 2) continue;
      double t = splits > 1 ? join + splits * part : 0.0;
      if (tile == 256) t += 11.0 + static_cast<double>((groups + 255) / 256) * each * 1.55;
      else if (groups <= 256) t += 5.0 + each * 0.82;
      else t += 5.0 + static_cast<double>((groups + 511) / 512) * each * 1.07;
      if (p.tile == 0 || t < best) {
        best = t;
        p.tile = tile;
        p.sp = Split{static_cast<int>(m), static_cast<int>(n), static_cast<int>(splits), each};
      }
    }
  }
  p.weight_bytes = p.sp.splits > 1 ? (static_cast<size_t>(p.sp.splits) * out * in * 4 + 255) / 256 * 256 : 0;
  p.bias_bytes = bias ? static_cast<size_t>(p.sp.splits) * p.sp.n_tiles * out * 4 : 0;
  return p;
}

// Copies to LDS need bf16 rows that start on 16 bytes, a turn of them within 2 GB.
bool copies_dy(const LinearArgs &a) {
  return a.dy_bf16 && reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 && a.lddy % 8 == 0 && (a.lddy * 64 + a.out) * 2 < 0x7fffffff;
}

Plan plan_of(const LinearArgs &a) { return plan_of(a.rows, a.out, a.in, a.dy_bf16, copies_dy(a), a.db != nullptr); }

float *weight_parts(const LinearArgs &a, const Plan &p) { return p.sp.splits > 1 ? static_cast<float *>(a.work) : nullptr; }
float *bias_parts(const LinearArgs &a, const Plan &p) {
  return a.db ? reinterpret_cast<float *>(static_cast<char *>(a.work) + p.weight_bytes) : nullptr;
}

template <int BM, int BN, int BK, int WM, int WN, typename T, int FMT, bool COPY>
void linear_one(const LinearArgs &a, const Plan &p, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.sp.m_tiles) * p.sp.n_tiles * p.sp.splits);
  linear_grad_kernel<BM, BN, BK, WM, WN, T, FMT, COPY><<<grid, 64 * WM * WN, 0, s>>>(a, p.sp, weight_parts(a, p), bias_parts(a, p));
}

template <typename T, int FMT>
void linear_few(const LinearArgs &a, hipStream_t s) {
  const int64_t quads = (a.in + 3) / 4;
  const dim3 grid(static_cast<unsigned>((a.out * quads + kBlock - 1) / kBlock));
  if (a.grad_bf16) linear_grad_few_kernel<T, uint16_t, FMT><<<grid, kBlock, 0, s>>>(a, static_cast<uint32_t>(quads));
  else linear_grad_few_kernel<T, float, FMT><<<grid, kBlock, 0, s>>>(a, static_cast<uint32_t>(quads));
}

template <int FMT>
void linear_by_type(const LinearArgs &a, const Plan &p, hipStream_t s) {
  if (a.rows < kFewRows) {
    if (a.dy_bf16) linear_few<uint16_t, FMT>(a, s);
    else linear_few<float, FMT>(a, s);
    return;
  }
  if (!a.dy_bf16) linear_one<128, 128, 32, 2, 2, float, FMT, false>(a, p, s);
  else if (!copies_dy(a)) linear_one<128, 128, 64, 2, 2, uint16_t, FMT, false>(a, p, s);
  else if (p.tile == 256) linear_one<256, 256, 64, 2, 4, uint16_t, FMT, true>(a, p, s);
  else linear_one<128, 128, 64, 2, 2, uint16_t, FMT, true>(a, p, s);
}

}  // namespace

bool linear_fits(int64_t rows, int64_t out, int64_t in) {
  // a turn's codes lie within 2 GB; a thread for every four elements, or 256 for a tile, fit the grid
  return in <= (int64_t{1} << 24) && out <= (int64_t{1} << 31) && rows <= (int64_t{1} << 24) &&
         out * ((in + 3) / 4) <= kMaxGrid * kBlock - kBlock && ((out + 127) / 128) * ((in + 127) / 128) <= kMaxGrid / 2;
}

size_t linear_work_bytes(int64_t rows, int64_t out, int64_t in, bool dy_bf16, bool bias) {
  // of the two plans that a call may take by dY's alignment, the larger
  const Plan p = plan_of(rows, out, in, dy_bf16, dy_bf16, bias), q = plan_of(rows, out, in, dy_bf16, false, bias);
  return std::max(p.weight_bytes + p.bias_bytes, q.weight_bytes + q.bias_bytes);
}

void launch_linear_grad(const LinearArgs &a, hipStream_t s) {
  const Plan p = plan_of(a);
  if (a.fmt == kE4M3) linear_by_type<kE4M3>(a, p, s);
  else linear_by_type<kInt8>(a, p, s);
}

bool linear_needs_join(const LinearArgs &a) { return a.rows >= kFewRows && (a.db != nullptr || plan_of(a).sp.splits > 1); }

void launch_linear_join(const LinearArgs &a, hipStream_t s) {
  const Plan p = plan_of(a);
  const auto blocks = [](int64_t n) { return (n + 4 * kBlock - 1) / (4 * kBlock); };
  const int64_t weight = p.sp.splits > 1 ? blocks(a.out * a.in) : 0, bias = a.db ? blocks(a.out) : 0;
  const dim3 grid(static_cast<unsigned>(weight + bias));
  const int64_t bias_count = static_cast<int64_t>(p.sp.splits) * p.sp.n_tiles;
  if (a.grad_bf16) join_kernel<uint16_t><<<grid, kBlock, 0, s>>>(a, weight_parts(a, p), p.sp.splits, weight, bias_parts(a, p), bias_count);
  else join_kernel<float><<<grid, kBlock, 0, s>>>(a, weight_parts(a, p), p.sp.splits, weight, bias_parts(a, p), bias_count);
}

}  // namespace ob
