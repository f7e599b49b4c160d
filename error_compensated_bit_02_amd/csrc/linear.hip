// A linear layer of the list (gfx950): its forward with bias, checkpoint,
// activation and residual, and the gradient to its input with the activation's
// derivative and an added gradient, each in the product's own epilogue.
//
//   forward   h[t][o] = sum over i of x[t][i] W[o][i] + b[o];  y = fn(h) + residual
//   backward  dx[t][i] = (sum over o of dy[t][o] W[o][i]) * fn'(kept[t][i]) + add[t][i]
//
// Both are one product C[t][f] = sum over k of B[t][k] A(f, k) on the bf16 matrix
// units with fp32 accumulators; B's rows lie along k, A's (the weight) along k in
// the forward and along f in the backward.  The weight is the instruction's first
// operand, so a lane's four results are four consecutive f of one token.
//
// fp32 operands are cut into three bf16 parts each (pack_kernel), rounded to
// nearest, so that each part is at most 2^-8 of the one before and they add up to
// the value exactly (but for bits below bf16's last, 2^-133).  Of two fp32 operands
// the products of parts whose order sums to at most 2 are taken, six of nine; the
// others are below 2^-25 of the product.  With one bf16 operand all three are taken
// and products are exact.
#include "internal.h"
#include "activation.h"
#include "act_math.h"
#include "tiles.h"

#include <algorithm>

#pragma clang fp contract(off)

namespace ob {
namespace {

constexpr int kTurn = 64;            // contraction steps of a turn
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

// What multiplies: matrices of bf16 parts whose rows start on 16 bytes.
struct Product {
  int64_t rows, features, depth;     // of C, and the contraction's length: a multiple of 8, past its true end B is zero
  int64_t a_rows;                    // backward: A's rows, the true length
  const uint16_t *a, *b;
  int64_t lda, ldb, a_part, b_part;  // row strides and distances of the parts, in elements
  int pairs;                         // products of parts
  uint32_t a_sel, b_sel;             // two bits a pair: the parts of each operand
};

// ---------------------------------------------------------------------------
// the epilogue: 32 tokens of FW features, from fp32 sums in LDS
// ---------------------------------------------------------------------------
// Eight consecutive elements of a row as fp32; absent ones are 0.
__device__ __forceinline__ void read8(const void *p, bool f32, bool vec, int n, float (&v)[8]) {
  if (vec && n >= 8) {
    if (f32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 w = static_cast<const f32x4 *>(p)[h];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * h + k] = w[k];
      }
    } else {
      const u32x4 w = *static_cast<const u32x4 *>(p);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = 0.0f;
    if (k < n) v[k] = f32 ? static_cast<const float *>(p)[k] : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[k]) << 16);
  }
}

__device__ __forceinline__ void write8(void *p, bool f32, bool vec, int n, const float (&v)[8]) {
  if (f32) {
    if (vec && n >= 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) static_cast<f32x4 *>(p)[h] = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
      return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) static_cast<float *>(p)[k] = v[k];
    return;
  }
  u32x4 w;
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
  if (vec && n >= 8) {
    *static_cast<u32x4 *>(p) = w;
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) static_cast<uint16_t *>(p)[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
}

__device__ __forceinline__ void write_bytes(uint8_t *p, int n, u32x2 w) {
  if (n >= 8) {
    *reinterpret_cast<u32x2 *>(p) = w;
    return;
  }
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (k < n) p[k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
}

template <bool FINE>
__device__ __forceinline__ void act8(int fn, float (&v)[8]) {
  if (fn == kActGelu) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = act_value<kActGelu, FINE>(v[k]);
  } else if (fn == kActGeluTanh) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = act_value<kActGeluTanh, FINE>(v[k]);
  } else if (fn == kActSilu) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = act_value<kActSilu, FINE>(v[k]);
  }
}

template <bool FINE>
__device__ __forceinline__ void slope8(int fn, const float (&x)[8], float (&v)[8]) {
  if (fn == kActGelu) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = v[k] * act_slope<kActGelu, FINE>(x[k]);
  } else if (fn == kActGeluTanh) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = v[k] * act_slope<kActGeluTanh, FINE>(x[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = v[k] * act_slope<kActSilu, FINE>(x[k]);
  }
}

// Row stride of the sums in LDS, in floats: 16 bytes more than a row.
template <int FW>
constexpr int kSlabRow = FW + 4;

// A wavefront turns the sums of tokens t0 .. t0 + 31 and features f0 .. f0 + FW - 1
// into results.  A lane has eight features of every RPI-th token.
template <int FW, bool BACK>
__device__ __forceinline__ void finish(const LayerArgs &a, OB_LDS const float *slab, int64_t t0, int64_t f0) {
  constexpr int LPR = FW / 8, RPI = 64 / LPR, NR = 32 / RPI;
  const int lane = threadIdx.x & 63, c = lane % LPR, r0 = lane / LPR;
  const int64_t f = f0 + c * 8;
  const int n = static_cast<int>(max(int64_t{0}, min(int64_t{8}, a.features - f)));
  const auto sums = [&](int j, float (&v)[8]) __attribute__((always_inline)) {
    OB_LDS const float *p = slab + (r0 + RPI * j) * kSlabRow<FW> + c * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 w = *(OB_LDS const f32x4 *)(p + 4 * h);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[4 * h + k] = w[k];
    }
  };
  float bias[8], scale[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) bias[k] = scale[k] = 0.0f;
  if constexpr (!BACK) {
    if (a.bias) read8(static_cast<const char *>(a.bias) + f * (a.weight_f32 ? 4 : 2), a.weight_f32, true, n, bias);
    if (a.codes) {
      uint32_t top[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) top[k] = 0;
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        if (t0 + r0 + RPI * j < a.rows) {
          float v[8];
          sums(j, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) top[k] = max(top[k], __float_as_uint(v[k] + bias[k]) & 0x7fffffffu);
        }
      }
#pragma unroll
      for (int d = LPR; d < 64; d <<= 1) {
#pragma unroll
        for (int k = 0; k < 8; ++k) top[k] = max(top[k], static_cast<uint32_t>(__shfl_xor(static_cast<int>(top[k]), d)));
      }
      u32x2 w = {0, 0};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t s = a.fmt == kE4M3 ? act_scale<kE4M3>(top[k]) : act_scale<kInt8>(top[k]);
        scale[k] = a.fmt == kE4M3 ? act_inverse<kE4M3>(s) : act_inverse<kInt8>(s);
        w[k >> 2] |= s << (8 * (k & 3));
      }
      if (r0 == 0 && t0 < a.rows) write_bytes(a.scales + t0 / kActBlock * a.pitch + f, n, w);
    }
  } else {
    if (a.fn != kActNone && n > 0 && t0 < a.rows) {    // whole groups of eight are in bounds, the pitch being a multiple of 64
      const u32x2 w = *reinterpret_cast<const u32x2 *>(a.scales + t0 / kActBlock * a.pitch + f);
#pragma unroll
      for (int k = 0; k < 8; ++k) scale[k] = act_scale_or_nan((w[k >> 2] >> (8 * (k & 3))) & 0xffu);
    }
  }
  if (n <= 0) return;
  const int es = a.f32 ? 4 : 2;
#pragma unroll 1
  for (int j = 0; j < NR; ++j) {
    const int64_t t = t0 + r0 + RPI * j;
    if (t >= a.rows) break;
    float v[8];
    sums(j, v);
    if constexpr (!BACK) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] + bias[k];
      if (a.codes) write_bytes(a.codes + t * a.pitch + f, n, a.fmt == kE4M3 ? encode8<kE4M3>(v, scale) : encode8<kInt8>(v, scale));
      if (a.f32) act8<true>(a.fn, v);
      else act8<false>(a.fn, v);
    } else if (a.fn != kActNone) {
      const u32x2 w = *reinterpret_cast<const u32x2 *>(a.codes + t * a.pitch + f);
      float x[8];
      if (a.fmt == kE4M3) decode8<kE4M3>(w, scale, x);
      else decode8<kInt8>(w, scale, x);
      if (a.f32) slope8<true>(a.fn, x, v);
      else slope8<false>(a.fn, x, v);
    }
    if (a.add) {
      float r[8];
      read8(static_cast<const char *>(a.add) + (t * a.ldadd + f) * es, a.f32, a.vec_add, n, r);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] + r[k];
    }
    write8(static_cast<char *>(a.y) + (t * a.ldy + f) * es, a.f32, a.vec_y, n, v);
  }
}

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------
// 16-byte unit u of row r of a tile whose rows are 128 bytes along k lies at unit
// u ^ swizzle_k(r): the 16 rows that one read touches at one k lie on all banks.
__device__ __forceinline__ int swizzle_k(int r) { return (r >> 1) & 7; }

// One workgroup's tile of C over one slice of the contraction: BF features, BT
// tokens, WF x WT wavefronts.  BACK: A lies along f.
//
// Stages.  A turn's two steps of 32 read their operands from LDS one step ahead of
// their products.  The barrier stands between them: behind it the next turn's tile
// is in LDS and nobody reads the present one any more, so the copies of the turn
// STAGES ahead go into its place.
template <int BF, int BT, int WF, int WT, int STAGES, bool BACK>
__global__ __launch_bounds__(64 * WF * WT, 2) void layer_kernel(const LayerArgs a, const Product q, const Split sp, float *part) {
  constexpr int NW = WF * WT, FI = BF / WF / 16, FO = BT / WT / 16, FW = FI * 16;
  constexpr int A_BYTES = BF * kTurn * 2, B_BYTES = BT * kTurn * 2, STAGE = A_BYTES + B_BYTES;
  constexpr int JA = A_BYTES / 1024 / NW, JB = B_BYTES / 1024 / NW, RA = 512 / BF;
  static_assert(JA * NW * 1024 == A_BYTES && JB * NW * 1024 == B_BYTES && FO % 2 == 0, "tile shape");
  static_assert(!BACK || BF >= 128, "the transposing read's swizzle spans eight units");
  static_assert(NW * 32 * kSlabRow<FW> * 4 <= STAGES * STAGE, "the epilogue's sums fit the stages");
  __shared__ __attribute__((aligned(1024))) unsigned char shared[STAGES * STAGE];
  OB_LDS unsigned char *const lds = (OB_LDS unsigned char *)shared;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wf = wave / WT, wt = wave % WT, g = lane >> 4, li = lane & 15;
  const Where at = where(sp);
  const int64_t f0 = static_cast<int64_t>(at.mt) * BF, t0 = static_cast<int64_t>(at.nt) * BT;
  const int turns_of_pair = static_cast<int>((q.depth + kTurn - 1) / kTurn);
  const int64_t first = at.split * sp.turns_each;
  const int turns = static_cast<int>(min(sp.turns_each, static_cast<int64_t>(turns_of_pair) * q.pairs - first));

  f32x4 acc[FI][FO];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int o = 0; o < FO; ++o) acc[i][o] = f32x4{0, 0, 0, 0};

  // Where this lane's 16 bytes of each copy come from: the copies write LDS in
  // lane order, so the swizzle is applied to the source.
  int from_a[JA], from_b[JB];
#pragma unroll
  for (int j = 0; j < JA; ++j) {
    if constexpr (BACK) {
      const int r = (wave * JA + j) * RA + lane / (BF / 8), c = lane % (BF / 8);
      from_a[j] = r * static_cast<int>(q.lda) * 2 + (((c >> 1) ^ swizzle_a(r)) << 5) + (c & 1) * 16;
    } else {
      const int r = (wave * JA + j) * 8 + (lane >> 3);
      from_a[j] = r * static_cast<int>(q.lda) * 2 + (((lane & 7) ^ swizzle_k(r)) << 4);
    }
  }
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    const int r = (wave * JB + j) * 8 + (lane >> 3);
    from_b[j] = r * static_cast<int>(q.ldb) * 2 + (((lane & 7) ^ swizzle_k(r)) << 4);
  }
  const int features = static_cast<int>(min(int64_t{BF}, q.features - f0)), tokens = static_cast<int>(min(int64_t{BT}, q.rows - t0));
  const int lda = static_cast<int>(q.lda), ldb = static_cast<int>(q.ldb);
  // the next turn to be copied: its pair, its place in the pair, how many are left
  int pair = static_cast<int>(first / turns_of_pair), kt = static_cast<int>(first % turns_of_pair), left = turns;

  const auto start = [&](OB_LDS unsigned char *dst) __attribute__((always_inline)) {
    const int64_t k0 = static_cast<int64_t>(kt) * kTurn;
    const int depth = static_cast<int>(min(int64_t{kTurn}, q.depth - k0)), any = -left >> 31;    // all ones or zeros by whether there is a turn
    const uint16_t *pa = q.a + ((q.a_sel >> (2 * pair)) & 3) * q.a_part, *pb = q.b + ((q.b_sel >> (2 * pair)) & 3) * q.b_part;
    pa += BACK ? k0 * q.lda + f0 : f0 * q.lda + k0;
    pb += t0 * q.ldb + k0;
    const auto ra = buffer(pa, (BACK ? ((static_cast<int>(min(int64_t{kTurn}, q.a_rows - k0)) - 1) * lda + static_cast<int>(q.features - f0)) * 2 : ((features - 1) * lda + depth) * 2) & any);
    const auto rb = buffer(pb, (((tokens - 1) * ldb + depth) * 2) & any);
    const bool cut = depth < kTurn;      // units past the contraction's end are read as past the buffer's
#pragma unroll
    for (int j = 0; j < JA; ++j) {
      int from = from_a[j];
      if constexpr (!BACK) {
        const int r = (wave * JA + j) * 8 + (lane >> 3);
        if (cut && ((lane & 7) ^ swizzle_k(r)) * 8 >= depth) from = 0x7ffffff0;
      }
      copy16(ra, dst + (wave * JA + j) * 1024, from);
    }
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      int from = from_b[j];
      const int r = (wave * JB + j) * 8 + (lane >> 3);
      if (cut && ((lane & 7) ^ swizzle_k(r)) * 8 >= depth) from = 0x7ffffff0;
      copy16(rb, dst + A_BYTES + (wave * JB + j) * 1024, from);
    }
    --left;
    if (++kt == turns_of_pair) {
      kt = 0;
      if (left > 0) ++pair;
    }
  };
  constexpr int kLoads = JA + JB;

  struct Operands {
    bf16x8 a[FI], b[FO];
  };
  const int row_a = 8 * g + (li >> 2), sw_a = (li >> 2) | (g & 1) << 2;     // of the transposing read
  const auto fetch = [&](OB_LDS const unsigned char *T, int kk, Operands &f) __attribute__((always_inline)) {
    const int unit = ((kk * 4 + g) ^ swizzle_k(li)) << 4;
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      if constexpr (BACK) {
        OB_LDS const unsigned char *p = T + (kk * 32 + row_a) * (BF * 2) + (((wf * FI + i) ^ sw_a) << 5) + (li & 3) * 8;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((OB_LDS s16x4 *)(p));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((OB_LDS s16x4 *)(p + 4 * BF * 2));
        f.a[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      } else {
        f.a[i] = *(OB_LDS const bf16x8 *)(T + ((wf * FI + i) * 16 + li) * (kTurn * 2) + unit);
      }
    }
#pragma unroll
    for (int o = 0; o < FO; ++o) f.b[o] = *(OB_LDS const bf16x8 *)(T + A_BYTES + ((wt * FO + o) * 16 + li) * (kTurn * 2) + unit);
  };
  const auto multiply = [&](const Operands &f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int o = 0; o < FO; ++o) acc[i][o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.a[i], f.b[o], acc[i][o], 0, 0, 0);
  };
  // Spreads the reads between the products: the wavefronts of a SIMD come out of
  // the barrier together, and a run of reads would fill the LDS queue while the
  // matrix unit stands still.
  const auto interleave = [&]() __attribute__((always_inline)) {
    constexpr int kReads = (BACK ? 2 : 1) * FI + FO;
#pragma unroll
    for (int k = 0; k < kReads; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one product
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one read
    }
  };
  // One turn: x holds its first step's operands, and the next turn's afterwards.
  // The two stages differ, which __restrict says: the compiler would otherwise
  // hold every read back until all copies have landed.
  const auto turn = [&](Operands &x, Operands &y, OB_LDS unsigned char *__restrict cur, OB_LDS unsigned char *__restrict next)
                        __attribute__((always_inline)) {
    fetch(cur, 1, y);
    multiply(x);
    interleave();
    __builtin_amdgcn_sched_barrier(0);
    wait_loads<(STAGES - 2) * kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    start(cur);
    fetch(next, 0, x);
    multiply(y);
    interleave();
    __builtin_amdgcn_sched_barrier(0);
  };

#pragma unroll
  for (int s = 0; s < STAGES; ++s) start(lds + s * STAGE);
  wait_loads<(STAGES - 1) * kLoads>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  {
    Operands x, y;
    fetch(lds, 0, x);
    int stage = 0;
    for (int t = 0; t < turns; ++t) {
      const int next = stage + 1 == STAGES ? 0 : stage + 1;
      turn(x, y, lds + stage * STAGE, lds + next * STAGE);
      stage = next;
    }
  }
  wait_loads<0>();                 // no copy may land after the workgroup has ended, or in the epilogue's sums

  if (part) {
    const int64_t ldp = (q.features + 3) / 4 * 4;
    float *out = part + at.split * q.rows * ldp;
#pragma unroll
    for (int o = 0; o < FO; ++o) {
      const int64_t t = t0 + (wt * FO + o) * 16 + li;
      if (t >= q.rows) continue;
#pragma unroll
      for (int i = 0; i < FI; ++i) {
        const int64_t f = f0 + (wf * FI + i) * 16 + g * 4;
        if (f < q.features) *reinterpret_cast<f32x4 *>(out + t * ldp + f) = acc[i][o];
      }
    }
    return;
  }
  __builtin_amdgcn_s_barrier();    // nobody reads the tiles any more
  asm volatile("" ::: "memory");
  OB_LDS float *slab = (OB_LDS float *)lds + wave * 32 * kSlabRow<FW>;
#pragma unroll
  for (int o = 0; o < FO; o += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < FI; ++i) *(OB_LDS f32x4 *)(slab + (h * 16 + li) * kSlabRow<FW> + i * 16 + g * 4) = acc[i][o + h];
    __builtin_amdgcn_wave_barrier();
    finish<FW, BACK>(a, slab, t0 + (wt * FO + o) * 16, f0 + wf * FW);
    __builtin_amdgcn_wave_barrier();
  }
}

// The slices' sums in order, and the epilogue: a wavefront takes 32 tokens of 64
// features.
constexpr int kJoinWidth = 64;
template <bool BACK>
__global__ __launch_bounds__(kBlock) void layer_join_kernel(const LayerArgs a, const float *part, int splits) {
  __shared__ __attribute__((aligned(16))) float shared[kWaves * 32 * kSlabRow<kJoinWidth>];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t across = static_cast<uint32_t>((a.features + kJoinWidth - 1) / kJoinWidth);
  const uint32_t id = blockIdx.x * kWaves + wave, band = id / across;
  const int64_t t0 = static_cast<int64_t>(band) * 32, f0 = static_cast<int64_t>(id - band * across) * kJoinWidth;
  if (t0 >= a.rows) return;
  const int64_t ldp = (a.features + 3) / 4 * 4, each = a.rows * ldp;
  OB_LDS float *slab = (OB_LDS float *)shared + wave * 32 * kSlabRow<kJoinWidth>;
  const int c = lane % 16, r0 = lane / 16;
  const int64_t f = f0 + c * 4;
#pragma unroll 2
  for (int j = 0; j < 8; ++j) {
    const int64_t t = t0 + r0 + 4 * j;
    f32x4 v = {0, 0, 0, 0};
    if (t < a.rows && f < a.features) {
      const float *p = part + t * ldp + f;
#pragma unroll 4
      for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4 *>(p + s * each);
    }
    *(OB_LDS f32x4 *)(slab + (r0 + 4 * j) * kSlabRow<kJoinWidth> + c * 4) = v;
  }
  __builtin_amdgcn_wave_barrier();
  finish<kJoinWidth, BACK>(a, slab, t0, f0);
}

// ---------------------------------------------------------------------------
// operands that the product cannot read as they are
// ---------------------------------------------------------------------------
// A matrix [rows][cols] as bf16 parts [PARTS][rows][pitch], pitch a multiple of 64
// and its end zero: fp32 as three parts, bf16 whose rows do not start on 16 bytes
// as one.
struct PackArgs {
  const void *from;
  int64_t ld;
  uint16_t *to;
  int64_t rows, cols, pitch;
};

// An fp32 value as three bf16 parts, each the rest rounded to nearest.  Values that
// would round to an infinity are cut instead; infinities and NaNs have no rest.
__device__ __forceinline__ void parts3(float x, uint16_t (&h)[3]) {
  const auto rounded = [](float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); };
  const uint32_t b = __float_as_uint(x);
  h[0] = rounded(x);
  if ((b & 0x7fffffffu) >= kInfBits) {
    h[1] = h[2] = 0;
    return;
  }
  if ((h[0] & 0x7fffu) == 0x7f80u) h[0] = static_cast<uint16_t>(b >> 16);
  const float r1 = x - __uint_as_float(static_cast<uint32_t>(h[0]) << 16);
  h[1] = rounded(r1);
  const float r2 = r1 - __uint_as_float(static_cast<uint32_t>(h[1]) << 16);
  h[2] = rounded(r2);
}

template <typename T>
__global__ __launch_bounds__(kBlock) void pack_kernel(const PackArgs a) {
  const int64_t units = a.pitch / 8, total = a.rows * units, step = static_cast<int64_t>(gridDim.x) * kBlock;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; id < total; id += step) {
    const int64_t r = id / units, c = (id - r * units) * 8;
    const T *p = static_cast<const T *>(a.from) + r * a.ld + c;
    T v[8];
    if (c + 8 <= a.cols) {
      __builtin_memcpy(v, p, sizeof(v));       // rows start anywhere
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = c + k < a.cols ? p[k] : T{0};
    }
    uint16_t *out = a.to + r * a.pitch + c;
    if constexpr (sizeof(T) == 2) {
      __builtin_memcpy(__builtin_assume_aligned(out, 16), v, 16);
    } else {
      uint16_t w[3][8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint16_t h[3];
        parts3(v[k], h);
#pragma unroll
        for (int s = 0; s < 3; ++s) w[s][k] = h[s];
      }
#pragma unroll
      for (int s = 0; s < 3; ++s) __builtin_memcpy(__builtin_assume_aligned(out + s * a.rows * a.pitch, 16), w[s], 16);
    }
  }
}

// ---------------------------------------------------------------------------
// plans
// ---------------------------------------------------------------------------
struct Tiles {
  int features, tokens;
};
constexpr Tiles kTiles[] = {{256, 256}, {128, 128}, {128, 32}};

int64_t up64(int64_t n) { return (n + 63) / 64 * 64; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int64_t features_of(const LayerShape &s) { return s.back ? s.in : s.out; }
int64_t depth_of(const LayerShape &s) { return s.back ? s.out : s.in; }

template <int BF, int BT, int WF, int WT, int STAGES>
void layer_one(const LayerArgs &a, const LayerPlan &p, const Product &q, float *part, hipStream_t s) {
  const Split sp{p.m_tiles, p.n_tiles, p.splits, p.turns_each};
  const dim3 grid(static_cast<unsigned>(p.m_tiles) * p.n_tiles * p.splits);
  if (a.shape.back) layer_kernel<BF, BT, WF, WT, STAGES, true><<<grid, 64 * WF * WT, 0, s>>>(a, q, sp, part);
  else layer_kernel<BF, BT, WF, WT, STAGES, false><<<grid, 64 * WF * WT, 0, s>>>(a, q, sp, part);
}

void pack(const void *from, bool f32, int64_t ld, int64_t rows, int64_t cols, void *to, hipStream_t s) {
  const PackArgs a{from, ld, static_cast<uint16_t *>(to), rows, cols, up64(cols)};
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((rows * (a.pitch / 8) + kBlock - 1) / kBlock, 1 << 16)));
  if (f32) pack_kernel<float><<<grid, kBlock, 0, s>>>(a);
  else pack_kernel<uint16_t><<<grid, kBlock, 0, s>>>(a);
}

char *work_at(const LayerArgs &a, size_t bytes) { return static_cast<char *>(a.work) + bytes; }

}  // namespace

bool layer_fits(int64_t rows, int64_t out, int64_t in) {
  // a tile's 256 rows (or 64 of the weight) lie within 2 GB; the large tiles fit the grid
  constexpr int64_t kMost = int64_t{1} << 21;
  return rows >= 0 && rows <= (int64_t{1} << 24) && out >= 1 && out <= kMost && in >= 1 && in <= kMost &&
         ((rows + 255) / 256) * ((std::max(out, in) + 255) / 256) <= kMaxGrid / 2;
}

LayerPlan layer_plan(const LayerShape &s) {
  LayerPlan p{};
  const int64_t features = features_of(s), depth = depth_of(s);
  p.a_parts = s.weight_f32 ? 3 : 1;
  p.b_parts = s.f32 ? 3 : 1;
  p.pack_a = s.weight_f32 || s.in % 8 != 0;
  p.pack_b = s.f32 || depth % 8 != 0 || !s.aligned;
  const int pairs = p.a_parts == 3 && p.b_parts == 3 ? 6 : std::max(p.a_parts, p.b_parts);
  const int64_t turns = (depth + kTurn - 1) / kTurn * pairs;
  if (p.pack_a) p.a_bytes = up256(static_cast<size_t>(p.a_parts) * s.out * up64(s.in) * 2);
  if (p.pack_b) p.b_bytes = up256(static_cast<size_t>(p.b_parts) * s.rows * up64(depth) * 2);
  const double part = static_cast<double>(s.rows) * features * 4 / 3e6;
  constexpr double kStart[] = {11.0, 5.0, 4.0}, kAlone[] = {1.6, 0.8, 0.45}, kFull[] = {1.6, 1.1, 0.6};
  constexpr int kPerCu[] = {1, 2, 2};
  double best = 0.0;
  p.tile = -1;
  for (int k = 0; k < 3; ++k) {
    const int64_t m = (features + kTiles[k].features - 1) / kTiles[k].features, n = (s.rows + kTiles[k].tokens - 1) / kTiles[k].tokens;
    const int64_t most = m * n >= 512 ? 1 : std::min<int64_t>(turns, 64);      // no slices where the tiles fill the card
    for (int64_t want = 1; want <= most; ++want) {
      const int64_t each = (turns + want - 1) / want, splits = (turns + each - 1) / each, groups = m * n * splits;
      if (splits != want || groups > kMaxGrid / 2) continue;
      double t = kStart[k] + (splits > 1 ? 4.0 + splits * part : 0.0);
      if (groups <= 256) t += each * kAlone[k];
      else t += static_cast<double>((groups + 256 * kPerCu[k] - 1) / (256 * kPerCu[k])) * each * kFull[k];
      if (p.tile < 0 || t < best) {
        best = t;
        p.tile = k;
        p.m_tiles = static_cast<int>(m);
        p.n_tiles = static_cast<int>(n);
        p.splits = static_cast<int>(splits);
        p.turns_each = each;
      }
    }
  }
  p.part_bytes = p.splits > 1 ? up256(static_cast<size_t>(p.splits) * s.rows * ((features + 3) / 4 * 4) * 4) : 0;
  return p;
}

void launch_layer_pack(const LayerArgs &a, const LayerPlan &p, hipStream_t s) {
  if (p.pack_a) pack(a.weight, a.weight_f32, a.shape.in, a.shape.out, a.shape.in, work_at(a, 0), s);
  if (p.pack_b) pack(a.x, a.f32, a.ldx, a.rows, depth_of(a.shape), work_at(a, p.a_bytes), s);
}

void launch_layer(const LayerArgs &a, const LayerPlan &p, hipStream_t s) {
  const int64_t depth = depth_of(a.shape);
  Product q{};
  q.rows = a.rows;
  q.features = a.features;
  q.depth = depth % 8 == 0 ? depth : up64(depth);      // then B is packed, and A too if it lies along k
  q.a_rows = depth;
  q.a = static_cast<const uint16_t *>(p.pack_a ? a.work : a.weight);
  q.lda = p.pack_a ? up64(a.shape.in) : a.shape.in;
  q.a_part = a.shape.out * q.lda;
  q.b = static_cast<const uint16_t *>(p.pack_b ? work_at(a, p.a_bytes) : a.x);
  q.ldb = p.pack_b ? up64(depth) : a.ldx;
  q.b_part = a.rows * q.ldb;
  if (p.a_parts == 3 && p.b_parts == 3) {      // small products first
    constexpr uint32_t kA[] = {2, 0, 1, 1, 0, 0}, kB[] = {0, 2, 1, 0, 1, 0};
    q.pairs = 6;
    for (int k = 0; k < 6; ++k) {
      q.a_sel |= kA[k] << (2 * k);
      q.b_sel |= kB[k] << (2 * k);
    }
  } else {
    q.pairs = std::max(p.a_parts, p.b_parts);
    for (int k = 0; k < q.pairs; ++k) {
      if (p.a_parts == 3) q.a_sel |= static_cast<uint32_t>(2 - k) << (2 * k);
      if (p.b_parts == 3) q.b_sel |= static_cast<uint32_t>(2 - k) << (2 * k);
    }
  }
  float *part = p.splits > 1 ? reinterpret_cast<float *>(work_at(a, p.a_bytes + p.b_bytes)) : nullptr;
  if (p.tile == 0) layer_one<256, 256, 4, 2, 2>(a, p, q, part, s);
  else if (p.tile == 1) layer_one<128, 128, 2, 2, 2>(a, p, q, part, s);
  else layer_one<128, 32, 4, 1, 4>(a, p, q, part, s);
}

void launch_layer_join(const LayerArgs &a, const LayerPlan &p, hipStream_t s) {
  const float *part = reinterpret_cast<const float *>(work_at(a, p.a_bytes + p.b_bytes));
  const int64_t waves = (a.rows + 31) / 32 * ((a.features + kJoinWidth - 1) / kJoinWidth);
  const dim3 grid(static_cast<unsigned>((waves + kWaves - 1) / kWaves));
  if (a.shape.back) layer_join_kernel<true><<<grid, kBlock, 0, s>>>(a, part, p.splits);
  else layer_join_kernel<false><<<grid, kBlock, 0, s>>>(a, part, p.splits);
}

}  // namespace ob
