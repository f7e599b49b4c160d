// A linear layer of the list (gfx950): its forward with bias, checkpoint,
// activation and residual, and the gradient to its input with the activation's
// derivative and an added gradient, each in the product's own epilogue.
//
//   forward   h[t][o] = sum over i of x[t][i] W[o][i] + b[o];  y = fn(h) + residual
//   backward  dx[t][i] = (sum over o of dy[t][o] W[o][i]) * fn'(kept[t][i]) + add[t][i]
//
// Both are one product C[t][f] = sum over k of B[t][k] A(f, k) on the bf16 matrix
// units with fp32 accumulators (a step aligns its addends to the largest and may cut what
// lies below 2^-24 of it: over 2048 products off by 2.7e-7 of a value of size 1, unbiased, a
// plain fp32 product by 3.9e-7); B's rows lie along k, A's (the weight) along k in
// the forward and along f in the backward.  The weight is the instruction's first
// operand, so a lane's four results are four consecutive f of one token.
//
// fp32 operands are cut into three bf16 parts each (pack_kernel, or on their way into
// LDS), rounded to nearest, so that each part is at most 2^-8 of the one before and
// they add up to the value exactly (but for bits below bf16's last, 2^-133).  Of two
// fp32 operands the products of parts whose order sums to at most 2 are taken, six of
// nine; the others are below 2^-25 of the product.  With one bf16 operand all three
// are taken and products are exact.
//
// What bounds it, measured on one card.  Large bf16 products: the matrix units at the
// clock that the card holds under them (about 1.8 GHz), 418 us for 16384 tokens of 2048 ->
// 8192 (1315 TFLOP/s; the library's product alone 375-391), 400 us for the gradient to
// the input of 8192 -> 2048 (1370; the library 435); of the 418, 55 are the copies beside
// the products.  fp32 at 4096^3: 640 us and 54 for the parts, 1290 TFLOP/s in six products.
// Few tokens: reading the weight (8192 x 8192 bf16 for one token 20.6 us, 6.5 TB/s).
// Between them, launches and the start and end of workgroups that have a CU to themselves.
#include "internal.h"
#include "activation.h"
#include "act_math.h"
#include "tiles.h"

#include <algorithm>
#include <type_traits>
#include <utility>

#pragma clang fp contract(off)

namespace ob {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

// What multiplies: bf16 matrices whose rows start on 16 bytes, or bf16 parts of fp32
// ones (pack_kernel), or fp32 matrices as they lie, cut on their way into LDS.
struct Product {
  int64_t rows, features, depth;     // of C, and the contraction's length: a multiple of 8, past its true end B is zero
  int64_t true_depth;
  const void *a, *b;
  int64_t lda, ldb, a_part, b_part;  // row strides and distances of the parts, in elements
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
      for (int h = 0; h < 2; ++h) __builtin_nontemporal_store(f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]}, static_cast<f32x4 *>(p) + h);
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
    __builtin_nontemporal_store(w, static_cast<u32x4 *>(p));
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) static_cast<uint16_t *>(p)[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
}

__device__ __forceinline__ void write_bytes(uint8_t *p, int n, u32x2 w) {
  if (n >= 8) {
    __builtin_nontemporal_store(w, reinterpret_cast<u32x2 *>(p));
    return;
  }
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (k < n) p[k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
}

// Row stride of the sums in LDS, in floats: 16 bytes more than a row.
template <int FW>
constexpr int kSlabRow = FW + 4;

// The largest of the lanes whose numbers differ in the bits from LANES on.
template <int LANES>
__device__ __forceinline__ uint32_t max_of_rows(uint32_t v) {
  if constexpr (LANES <= 4) v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x124, 0xf, 0xf, true)));   // rotations
  if constexpr (LANES <= 8) v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x128, 0xf, 0xf, true)));   // of 16 lanes
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

// The activation and its slope for bf16 results.  gelu_tanh's in fewer instructions
// than the checkpoint's kernels take, whose time is the memory's: the exponent
// as x (A + B x^2) and sigma' as s - s^2 (s is in [0, 1], so what cancels there is
// below 2^-24 of the slope's terms; backward of 8192 -> 2048 over 16384 tokens 471 us
// against 490).
constexpr float kTanhA = -2.302208198144325f, kTanhB = -0.1029432395800235f;   // -2 sqrt(2/pi) log2(e), times 0.044715
__device__ __forceinline__ float tanh_sigma(float x) {
  return reciprocal<false>(1.0f + __builtin_amdgcn_exp2f(x * __builtin_fmaf(x * x, kTanhB, kTanhA)));
}
template <int FN>
__device__ __forceinline__ float short_value(float x) {
  if constexpr (FN == kActGeluTanh) return x * tanh_sigma(x);
  else return act_value<FN, false>(x);
}
template <int FN>
__device__ __forceinline__ float short_slope(float x) {
  if constexpr (FN == kActGeluTanh) {
    const float s = tanh_sigma(x), ds = __builtin_fmaf(-s, s, s);
    const float c = __builtin_amdgcn_fmed3f(x, -64.0f, 64.0f);     // where ds is 0 the factor beside it stays finite
    return __builtin_fmaf(ds * c, __builtin_fmaf(c * c, 3.0f * kGeluK * kGeluC, kGeluC), s);
  } else {
    return act_slope<FN, false>(x);
  }
}

// What a wavefront's epilogue reads of 32 tokens beside the sums, as bf16 vectors
// and codes: loaded before the sums of the block in front are worked on, for a
// load's latency has nothing else to hide behind in a workgroup that ends.
template <int FW>
struct Beside {
  static constexpr int kLanes = FW / 8, kStep = 64 / kLanes, kRows = 32 / kStep;   // lanes of a token, tokens apart, tokens of a lane
  u32x4 add[kRows];
  u32x2 codes[kRows], scales;
};

template <int FW, bool BACK, int FN>
__device__ __forceinline__ void load_beside(const LayerArgs &a, int64_t t0, int64_t f0, Beside<FW> &b) {
  using B = Beside<FW>;
  const int lane = threadIdx.x & 63, r0 = lane / B::kLanes;
  const int64_t f = f0 + lane % B::kLanes * 8;
  const bool add = a.add && a.vec_add && !a.f32 && f + 8 <= a.features;
  b.scales = u32x2{0, 0};
  if (BACK && FN != kActNone && f < a.features && t0 < a.rows)    // whole groups of eight are in bounds, the pitch being a multiple of 64
    b.scales = *reinterpret_cast<const u32x2 *>(a.scales + t0 / kActBlock * a.pitch + f);
#pragma unroll
  for (int j = 0; j < B::kRows; ++j) {
    const int64_t t = t0 + r0 + B::kStep * j;
    if (t >= a.rows) continue;
    if (add) b.add[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.add) + t * a.ldadd + f));
    if (BACK && FN != kActNone && f < a.features) b.codes[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(a.codes + t * a.pitch + f));
  }
}

// A wavefront turns the sums of tokens t0 .. t0 + 31 and features f0 .. f0 + FW - 1
// into results.  A lane has eight features of every kStep-th token.
template <int FW, bool BACK, int FN>
__device__ __forceinline__ void finish(const LayerArgs &a, OB_LDS const float *slab, int64_t t0, int64_t f0, const Beside<FW> &b) {
  using B = Beside<FW>;
  const int lane = threadIdx.x & 63, c = lane % B::kLanes, r0 = lane / B::kLanes;
  const int64_t f = f0 + c * 8;
  const int n = static_cast<int>(max(int64_t{0}, min(int64_t{8}, a.features - f)));
  const auto sums = [&](int j, float (&v)[8]) __attribute__((always_inline)) {
    OB_LDS const float *p = slab + (r0 + B::kStep * j) * kSlabRow<FW> + c * 8;
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
      for (int j = 0; j < B::kRows; ++j) {
        float v[8];
        sums(j, v);
        const bool in = t0 + r0 + B::kStep * j < a.rows;
#pragma unroll
        for (int k = 0; k < 8; ++k) top[k] = max(top[k], in ? __float_as_uint(v[k] + bias[k]) & 0x7fffffffu : 0u);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) top[k] = max_of_rows<B::kLanes>(top[k]);
      u32x2 w = {0, 0};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t s = a.fmt == kE4M3 ? act_scale<kE4M3>(top[k]) : act_scale<kInt8>(top[k]);
        scale[k] = a.fmt == kE4M3 ? act_inverse<kE4M3>(s) : act_inverse<kInt8>(s);
        w[k >> 2] |= s << (8 * (k & 3));
      }
      if (r0 == 0 && t0 < a.rows) write_bytes(a.scales + t0 / kActBlock * a.pitch + f, n, w);
    }
  } else if constexpr (FN != kActNone) {
#pragma unroll
    for (int k = 0; k < 8; ++k) scale[k] = act_scale_or_nan((b.scales[k >> 2] >> (8 * (k & 3))) & 0xffu);
  }
  if (n <= 0) return;
  const int es = a.f32 ? 4 : 2;
#pragma unroll
  for (int j = 0; j < B::kRows; ++j) {
    const int64_t t = t0 + r0 + B::kStep * j;
    if (t >= a.rows) continue;
    float v[8];
    sums(j, v);
    if constexpr (!BACK) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] + bias[k];
      if (a.codes) write_bytes(a.codes + t * a.pitch + f, n, a.fmt == kE4M3 ? encode8<kE4M3>(v, scale) : encode8<kInt8>(v, scale));
      if constexpr (FN != kActNone) {
        if (a.f32) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = act_value<FN, true>(v[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = short_value<FN>(v[k]);
        }
      }
    } else if constexpr (FN != kActNone) {
      float x[8];
      if (a.fmt == kE4M3) decode8<kE4M3>(b.codes[j], scale, x);
      else decode8<kInt8>(b.codes[j], scale, x);
      if (a.f32) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = v[k] * act_slope<FN, true>(x[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = v[k] * short_slope<FN>(x[k]);
      }
    }
    if (a.add) {
      float r[8];
      if (a.vec_add && !a.f32 && n >= 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          r[2 * k] = __uint_as_float(b.add[j][k] << 16);
          r[2 * k + 1] = __uint_as_float(b.add[j][k] & 0xffff0000u);
        }
      } else {
        read8(static_cast<const char *>(a.add) + (t * a.ldadd + f) * es, a.f32, a.vec_add, n, r);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] + r[k];
    }
    write8(static_cast<char *>(a.y) + (t * a.ldy + f) * es, a.f32, a.vec_y, n, v);
  }
}

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------
// 16-byte unit u of row r of a tile whose rows lie along k, KT steps each, lies at
// unit u ^ swizzle_k(r): the 16 rows that one read touches at one k lie on all banks.
template <int KT>
__device__ __forceinline__ int swizzle_k(int r) { return KT == 64 ? (r >> 1) & 7 : (r >> 2) & 3; }

// f(0), f(1), ... f(N - 1) with constants.
template <typename F, int... I>
__device__ __forceinline__ void each(F &&f, std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }
template <int N, typename F>
__device__ __forceinline__ void each(F &&f) { each(f, std::make_integer_sequence<int, N>{}); }

// The products of two operands' parts that are taken, the small ones first.
constexpr int kPartA[] = {2, 0, 1, 1, 0, 0}, kPartB[] = {0, 2, 1, 0, 1, 0};

// One workgroup's tile of C over one slice of the contraction: BF features, BT
// tokens, WF x WT wavefronts, PA and PB parts of the operands.  BACK: A lies along f.
//
// Stages.  The operands of a step of 32 are read from LDS one step ahead of their
// products.  A turn's barrier stands where its last operands have been read: behind
// it the next turn's tile is in LDS and nobody reads the present one any more, so the
// copies of the turn STAGES ahead go into its place.
// Parts: all products of a step run on the same reads, so a part is loaded once a tile
// and not once a product.
// RAW: parts are cut from fp32 on the way into LDS instead of being read from a copy.
//
// Tiles.  256 x 256 on eight wavefronts of 64 x 128, two stages of 64: a byte of LDS is
// read for the fewest products, and the 128 sums a lane leave room for two steps'
// operands.  At 16384 x 2048 -> 8192, 418 us: 128 x 128 tiles 532, four wavefronts of
// 128 x 128 552, 128 x 256 on half a CU 530-540, five stages of 32 550, 32 x 32 x 16
// products 480-495, 256 lasting workgroups 505.  Copies in the first half of a step's
// products 418, over all of them 460, in a burst 451; no fences 460.
template <int BF, int BT, int WF, int WT, int KT, int PA, int PB, bool RAW, int STAGES, int WGS, bool BACK, int FN>
__global__ __launch_bounds__(64 * WF * WT, WGS * WF * WT / 4) void layer_kernel(const LayerArgs a, const Product q, const Split sp, float *part) {
  constexpr int NW = WF * WT, FI = BF / WF / 16, FO = BT / WT / 16, FW = FI * 16;      // fragments of a wavefront
  constexpr int UNITS = KT / 8, ROWS = 64 / UNITS;       // units of a row, rows of one copy
  constexpr int A_PART = BF * KT * 2, B_PART = BT * KT * 2, A_BYTES = PA * A_PART, STAGE = A_BYTES + PB * B_PART;
  constexpr int JA = A_PART / 1024 / NW, JB = B_PART / 1024 / NW, RA = 512 / BF;
  // RAW: fp32 operands pass through registers, UA and UB units of eight elements a lane
  constexpr bool RAW_A = RAW && PA == 3, RAW_B = RAW && PB == 3;
  constexpr int NT = 64 * NW, UA = RAW_A ? BF * KT / 8 / NT : 0, UB = RAW_B ? BT * KT / 8 / NT : 0, U = UA + UB;
  static_assert(JA * NW * 1024 == A_PART && JB * NW * 1024 == B_PART && FO % 2 == 0, "tile shape");
  static_assert(U == 0 || (KT == 32 && STAGES == 2), "a unit is cut a turn ahead of its products");
  static_assert(!BACK || BF >= 128, "the transposing read's swizzle spans eight units");
  static_assert(NW * 32 * kSlabRow<FW> * 4 <= STAGES * STAGE, "the epilogue's sums fit the stages");
  static_assert(WGS * STAGES * STAGE <= 160 * 1024, "LDS of a CU");
  __shared__ __attribute__((aligned(1024))) unsigned char shared[STAGES * STAGE];
  OB_LDS unsigned char *const lds = (OB_LDS unsigned char *)shared;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wf = wave / WT, wt = wave % WT, g = lane >> 4, li = lane & 15;
  const Where at = where(sp);
  const int64_t f0 = static_cast<int64_t>(at.mt) * BF, t0 = static_cast<int64_t>(at.nt) * BT;
  const int64_t first = at.split * sp.turns_each;
  const int turns = static_cast<int>(min(sp.turns_each, (q.true_depth + KT - 1) / KT - first));

  f32x4 acc[FI][FO];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int o = 0; o < FO; ++o) acc[i][o] = f32x4{};

  // Where this lane's 16 bytes of each copy come from: the copies write LDS in
  // lane order, so the swizzle is applied to the source.
  const auto row_of = [&](int copy) __attribute__((always_inline)) { return copy * ROWS + lane / UNITS; };
  const auto unit_of = [&](int copy) __attribute__((always_inline)) { return (lane % UNITS) ^ swizzle_k<KT>(row_of(copy)); };
  int from_a[JA], from_b[JB];
#pragma unroll
  for (int j = 0; j < JA; ++j) {
    if constexpr (BACK) {
      const int r = (wave * JA + j) * RA + lane / (BF / 8), c = lane % (BF / 8);
      from_a[j] = r * static_cast<int>(q.lda) * 2 + (((c >> 1) ^ swizzle_a(r)) << 5) + (c & 1) * 16;
    } else {
      from_a[j] = row_of(wave * JA + j) * static_cast<int>(q.lda) * 2 + unit_of(wave * JA + j) * 16;
    }
  }
#pragma unroll
  for (int j = 0; j < JB; ++j) from_b[j] = row_of(wave * JB + j) * static_cast<int>(q.ldb) * 2 + unit_of(wave * JB + j) * 16;
  const int features = static_cast<int>(min(int64_t{BF}, q.features - f0)), tokens = static_cast<int>(min(int64_t{BT}, q.rows - t0));
  const int lda = static_cast<int>(q.lda), ldb = static_cast<int>(q.ldb);
  // The next turn to be copied: where it reads, how much of the contraction is left,
  // and how many turns.
  const int64_t k0 = first * KT;
  const char *at_a = static_cast<const char *>(q.a) + (BACK ? k0 * q.lda + f0 : f0 * q.lda + k0) * 2;
  const char *at_b = static_cast<const char *>(q.b) + (t0 * q.ldb + k0) * 2;
  int left = turns, depth = static_cast<int>(q.depth - k0), a_rows = static_cast<int>(q.true_depth - k0);

  // The copies of a turn: their buffers and offsets, then the copies one by one.
  // Units past the contraction's end are read as past the buffer's.
  struct Turn {
    __amdgpu_buffer_rsrc_t a[PA], b[PB];
    int from_a[JA], from_b[JB];
  };
  const auto aim = [&](Turn &n) __attribute__((always_inline)) {
    const int any = -left >> 31;     // all ones or zeros by whether there is a turn
    const int steps = min(depth, KT), rows = min(a_rows, KT);
    const auto inside = [&](int copy, int from) __attribute__((always_inline)) { return unit_of(copy) * 8 < steps ? from : 0x7ffffff0; };
    if constexpr (!RAW_A) {
      const int size = (BACK ? (rows - 1) * lda + static_cast<int>(q.features - f0) : (features - 1) * lda + steps) * 2;
#pragma unroll
      for (int s = 0; s < PA; ++s) n.a[s] = buffer(at_a + s * q.a_part * 2, size & any);
#pragma unroll
      for (int j = 0; j < JA; ++j) n.from_a[j] = BACK ? from_a[j] : inside(wave * JA + j, from_a[j]);
    }
    if constexpr (!RAW_B) {
      const int size = ((tokens - 1) * ldb + steps) * 2;
#pragma unroll
      for (int s = 0; s < PB; ++s) n.b[s] = buffer(at_b + s * q.b_part * 2, size & any);
#pragma unroll
      for (int j = 0; j < JB; ++j) n.from_b[j] = inside(wave * JB + j, from_b[j]);
    }
    --left;
    depth -= KT;
    a_rows -= KT;
    at_a += BACK ? static_cast<int64_t>(lda) * (KT * 2) : KT * 2;
    at_b += KT * 2;
  };
  constexpr int kCopiesA = RAW_A ? 0 : PA * JA, kLoads = kCopiesA + (RAW_B ? 0 : PB * JB);
  const auto copy = [&](const Turn &n, int c, OB_LDS unsigned char *dst) __attribute__((always_inline)) {
    if (c < kCopiesA) {
      copy16(n.a[c / JA], dst + c / JA * A_PART + (wave * JA + c % JA) * 1024, n.from_a[c % JA]);
    } else {
      const int d = c - kCopiesA;
      copy16(n.b[d / JB], dst + A_BYTES + d / JB * B_PART + (wave * JB + d % JB) * 1024, n.from_b[d % JB]);
    }
  };

  // RAW: fp32 operands.  Rows past the end are read as the last one (their results are
  // dropped); of a row that ends within a unit the rest is 0, and so are the weight's
  // rows past the contraction's end.  raw_k: the first k of the turn to be read.
  float raw[U > 0 ? U : 1][8];
  int64_t raw_k = k0;
  int raw_left = turns;
  const auto fill = [&](int u) __attribute__((always_inline)) {
    const bool is_a = u < UA, along_f = BACK && is_a;
    const int id = static_cast<int>(threadIdx.x) + (is_a ? u : u - UA) * NT;
    const float *p;
    int64_t n;
    if (along_f) {
      const int64_t k = raw_k + id / (BF / 8), f = f0 + id % (BF / 8) * 8;
      p = static_cast<const float *>(q.a) + min(k, q.true_depth - 1) * q.lda + f;
      n = k < q.true_depth ? q.features - f : 0;
    } else {
      const int64_t k = raw_k + id % 4 * 8, r = id / 4;
      if (is_a) p = static_cast<const float *>(q.a) + min(f0 + r, q.features - 1) * q.lda + k;
      else p = static_cast<const float *>(q.b) + min(t0 + r, q.rows - 1) * q.ldb + k;
      n = q.true_depth - k;
    }
    if (n >= 8) {
      __builtin_memcpy(raw[u], p, sizeof(raw[u]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) raw[u][k] = k < n ? p[k] : 0.0f;
    }
  };
  // Two elements as three parts each, every part the rest rounded to nearest: the first
  // is held to the finite range, so a value past bf16's largest is its and its rest.
  const auto cut = [&](float x, float y, uint32_t (&w)[3]) __attribute__((always_inline)) {
    constexpr float kMost = 3.3895313892515355e38f;
    float px = __builtin_amdgcn_fmed3f(x, -kMost, kMost), py = __builtin_amdgcn_fmed3f(y, -kMost, kMost);
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      w[s] = pack_bf16(px, py);
      x = x - __uint_as_float(w[s] << 16);
      y = y - __uint_as_float(w[s] & 0xffff0000u);
      px = x;
      py = y;
    }
  };
  uint32_t parts[3][4];              // of the unit that is being cut
  const auto cut_pair = [&](int u, int pair) __attribute__((always_inline)) {
    uint32_t w[3];
    cut(raw[u][2 * pair], raw[u][2 * pair + 1], w);
#pragma unroll
    for (int s = 0; s < 3; ++s) parts[s][pair] = w[s];
  };
  const auto settle = [&](int u, OB_LDS unsigned char *dst) __attribute__((always_inline)) {
    const bool is_a = u < UA;
    const int id = static_cast<int>(threadIdx.x) + (is_a ? u : u - UA) * NT;
    int at_lds;
    if (BACK && is_a) {
      const int k = id / (BF / 8), c = id % (BF / 8);
      at_lds = k * (BF * 2) + (((c >> 1) ^ swizzle_a(k)) << 5) + (c & 1) * 16;
    } else {
      const int r = id / 4;
      at_lds = (is_a ? 0 : A_BYTES) + r * 64 + (((id % 4) ^ swizzle_k<32>(r)) << 4);
    }
#pragma unroll
    for (int s = 0; s < 3; ++s)
      *(OB_LDS u32x4 *)(dst + at_lds + s * (is_a ? A_PART : B_PART)) = u32x4{parts[s][0], parts[s][1], parts[s][2], parts[s][3]};
  };
  const auto next_raw = [&]() __attribute__((always_inline)) {
    raw_k += KT;
    --raw_left;
  };

  struct Operands {                // of a step of 32
    bf16x8 a[PA][FI], b[PB][FO];
  };
  // Of the transposing read, which gives a lane four k of its feature: where it starts for the wavefront's first
  // fragment; the others' units differ in the bits that the swizzle exchanges.
  const int row_a = 8 * g + (li >> 2), off_a = row_a * (BF * 2) + (((wf * FI) ^ swizzle_a(row_a)) << 5) + (li & 3) * 8;
  constexpr int kReads = PA * FI + PB * FO;                          // reads of a step
  const auto read = [&](OB_LDS const unsigned char *T, int kk, int r, Operands &f) __attribute__((always_inline)) {
    const int unit = ((kk * 4 + g) ^ swizzle_k<KT>(li)) << 4;
    if (r < PA * FI) {
      const int s = r / FI, i = r % FI;
      if constexpr (BACK) {
        OB_LDS const unsigned char *p = T + (off_a ^ (i << 5)) + s * A_PART + kk * 32 * (BF * 2);
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((OB_LDS s16x4 *)(p));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((OB_LDS s16x4 *)(p + 4 * BF * 2));
        f.a[s][i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      } else {
        f.a[s][i] = *(OB_LDS const bf16x8 *)(T + s * A_PART + ((wf * FI + i) * 16 + li) * (KT * 2) + unit);
      }
    } else {
      const int s = (r - PA * FI) / FO, o = (r - PA * FI) % FO;
      f.b[s][o] = *(OB_LDS const bf16x8 *)(T + A_BYTES + s * B_PART + ((wt * FO + o) * 16 + li) * (KT * 2) + unit);
    }
  };
  // One step: its products, with the reads of the next
  // step's operands and the copies spread between them: a run of either would fill its
  // queue, and a wavefront that waits there issues no products.  The fences keep the
  // compiler from gathering them again.
  constexpr int kProducts = PA == 3 && PB == 3 ? 6 : PA * PB, kOne = FI * FO, kMul = kProducts * kOne;
  constexpr int kSpan = (kMul + 1) / 2;          // reads and copies come with the first half of the products: the next barrier waits for both
  const auto step = [&](const Operands &x, OB_LDS const unsigned char *from, int kk, Operands &y, auto copies, const Turn &n,
                        OB_LDS unsigned char *dst) __attribute__((always_inline)) {
    each<kMul>([&](auto at) __attribute__((always_inline)) {
      constexpr int m = at, p = m / kOne, i = m % kOne / FO, o = m % FO;
      constexpr int s = kProducts == 6 ? kPartA[p] : PA == 3 ? 2 - p : 0, u = kProducts == 6 ? kPartB[p] : PB == 3 ? 2 - p : 0;
      acc[i][o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.a[s][i], x.b[u][o], acc[i][o], 0, 0, 0);
      constexpr int r0 = m < kSpan ? m * kReads / kSpan : kReads, r1 = m < kSpan ? (m + 1) * kReads / kSpan : kReads;
      each<r1 - r0>([&](auto r) __attribute__((always_inline)) { read(from, kk, r0 + r, y); });
      if constexpr (decltype(copies)::value) {
        constexpr int c0 = m < kSpan ? m * kLoads / kSpan : kLoads, c1 = m < kSpan ? (m + 1) * kLoads / kSpan : kLoads;
        each<c1 - c0>([&](auto c) __attribute__((always_inline)) { copy(n, c0 + c, dst); });
        // what is in registers is cut into the stage, four pairs a unit, by three quarters of the products, then read anew
        constexpr int kCut = kMul * 3 / 4, p0 = m < kCut ? m * 4 * U / kCut : 4 * U, p1 = m < kCut ? (m + 1) * 4 * U / kCut : 4 * U;
        each<p1 - p0>([&](auto pair) __attribute__((always_inline)) {
          constexpr int at_pair = p0 + pair;
          cut_pair(at_pair / 4, at_pair % 4);
          if constexpr (at_pair % 4 == 3) settle(at_pair / 4, dst);
        });
        if constexpr (U > 0 && m == kCut) {
          if (raw_left > 0) each<U>([&](auto u) __attribute__((always_inline)) { fill(u); });
          next_raw();
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  const auto arrived = [&]() __attribute__((always_inline)) {
    if constexpr (kLoads > 0) wait_loads<(STAGES - 2) * kLoads>();
    else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // One turn.  The two stages differ, which __restrict says: the compiler would
  // otherwise hold every read back until all copies have landed.
  // Two steps: x holds the first one's operands, and the next turn's afterwards.
  const auto turn_of_two = [&](Operands &x, Operands &y, OB_LDS unsigned char *__restrict cur, OB_LDS unsigned char *__restrict next)
                               __attribute__((always_inline)) {
    Turn n;
    step(x, cur, 1, y, std::false_type{}, n, cur);
    aim(n);
    arrived();
    step(y, next, 0, x, std::true_type{}, n, cur);
  };
  // One step: x holds its operands, y the next turn's afterwards.
  const auto turn_of_one = [&](Operands &x, Operands &y, OB_LDS unsigned char *__restrict cur, OB_LDS unsigned char *__restrict next)
                               __attribute__((always_inline)) {
    Turn n;
    aim(n);
    arrived();
    step(x, next, 0, y, std::true_type{}, n, cur);
  };

#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
    Turn n;
    aim(n);
#pragma unroll
    for (int c = 0; c < kLoads; ++c) copy(n, c, lds + s * STAGE);
    if constexpr (U > 0) {
      if (raw_left > 0) {
        each<U>([&](auto u) __attribute__((always_inline)) { fill(u); });
        each<U>([&](auto u) __attribute__((always_inline)) {
          each<4>([&](auto pair) __attribute__((always_inline)) { cut_pair(u, pair); });
          settle(u, lds + s * STAGE);
        });
      }
      next_raw();
    }
  }
  if constexpr (U > 0) {
    if (raw_left > 0) each<U>([&](auto u) __attribute__((always_inline)) { fill(u); });
    next_raw();
  }
  if constexpr (U > 0) wait_loads<0>();
  else wait_loads<(STAGES - 1) * kLoads>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  {
    Operands x, y;
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(lds, 0, r, x);
    int stage = 0;
    const auto stages = [&](auto &&turn, Operands &x, Operands &y) __attribute__((always_inline)) {
      const int next = stage + 1 == STAGES ? 0 : stage + 1;
      turn(x, y, lds + stage * STAGE, lds + next * STAGE);
      stage = next;
    };
    if constexpr (KT == 64) {
      for (int t = 0; t < turns; ++t) stages(turn_of_two, x, y);
    } else {
      // in pairs without a way out between them, past which the compiler would move the reads
      for (int t = turns / 2; t > 0; --t) {
        stages(turn_of_one, x, y);
        stages(turn_of_one, y, x);
      }
      if (turns % 2) stages(turn_of_one, x, y);
    }
  }
  wait_loads<0>();                 // no copy may land after the workgroup has ended, or in the epilogue's sums

  // A lane's sums: four features of one token of a fragment.
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
  const int64_t mine = t0 + wt * FO * 16, at_f = f0 + wf * FW;
  Beside<FW> beside[2];
  load_beside<FW, BACK, FN>(a, mine, at_f, beside[0]);
  __builtin_amdgcn_s_barrier();    // nobody reads the tiles any more
  asm volatile("" ::: "memory");
  OB_LDS float *slab = (OB_LDS float *)lds + wave * 32 * kSlabRow<FW>;
#pragma unroll
  for (int o = 0; o < FO; o += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < FI; ++i) *(OB_LDS f32x4 *)(slab + (h * 16 + li) * kSlabRow<FW> + i * 16 + g * 4) = acc[i][o + h];
    if (o + 2 < FO) load_beside<FW, BACK, FN>(a, mine + (o + 2) * 16, at_f, beside[(o / 2 + 1) & 1]);
    __builtin_amdgcn_wave_barrier();
    finish<FW, BACK, FN>(a, slab, mine + o * 16, at_f, beside[(o / 2) & 1]);
    __builtin_amdgcn_wave_barrier();
  }
}

// The slices' sums and the epilogue: a workgroup adds up 32 tokens of 32 features, four
// features a work-item, and its first wavefront finishes them.  Small blocks, as few
// tokens in many slices wait for one load after the other: 6-8 us where a wavefront
// with a block of its own took 20 (32 tokens of 1024 features in 32 slices).
constexpr int kJoinWidth = 32;
template <bool BACK, int FN>
__global__ __launch_bounds__(kBlock) void layer_join_kernel(const LayerArgs a, const float *part, int splits) {
  __shared__ __attribute__((aligned(16))) float shared[32 * kSlabRow<kJoinWidth>];
  OB_LDS float *slab = (OB_LDS float *)shared;
  const uint32_t across = static_cast<uint32_t>((a.features + kJoinWidth - 1) / kJoinWidth);
  const uint32_t band = blockIdx.x / across;
  const int64_t t0 = static_cast<int64_t>(band) * 32, f0 = static_cast<int64_t>(blockIdx.x - band * across) * kJoinWidth;
  const int64_t ldp = (a.features + 3) / 4 * 4, each = a.rows * ldp;
  const int r = threadIdx.x / 8, c = threadIdx.x % 8 * 4;
  Beside<kJoinWidth> beside;
  if (threadIdx.x < 64) load_beside<kJoinWidth, BACK, FN>(a, t0, f0, beside);
  f32x4 v = {0, 0, 0, 0};
  if (t0 + r < a.rows && f0 + c < a.features) {
    const float *p = part + (t0 + r) * ldp + f0 + c;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4 *>(p + s * each);
  }
  *(OB_LDS f32x4 *)(slab + r * kSlabRow<kJoinWidth> + c) = v;
  __syncthreads();
  if (threadIdx.x < 64) finish<kJoinWidth, BACK, FN>(a, slab, t0, f0, beside);
}

// ---------------------------------------------------------------------------
// a few tokens: bound by reading the weight
// ---------------------------------------------------------------------------
// Up to kLayerFew tokens are multiplied on the vector units in fp32, straight from
// the weight as it lies in the list, whatever its type or alignment: no copies of
// parts, no tile that is mostly padding, and in the forward no join.  One token of
// 1024 -> 4096 in bf16 7.5 us a call (the kernel 3.5), 13 through a tile of the matrix
// units; where these win, few_by_vectors says.
constexpr int kFewRows = 4;           // forward: features of a wavefront
constexpr int kFewLanes = 4;          // backward: lanes, of eight features each, of a workgroup
constexpr int kFewBlock = 512, kFewGroups = kFewBlock / kFewLanes;
constexpr int kFewEach = 8;           // backward: rows of a group, under way together with the others'
static_assert(kFewEach * kFewGroups == kLayerSlice, "a workgroup's rows are a slice");

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// Eight elements of a row as they lie, from anywhere; the last of a row one by one.
template <typename T>
struct Eight {
  T v[8];
  __device__ __forceinline__ void load(const T *p) { __builtin_memcpy(v, p, sizeof(v)); }
  __device__ __forceinline__ void load_some(const T *p, int64_t n) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? p[k] : T{0};
  }
  __device__ __forceinline__ float operator[](int k) const { return to_f32(v[k]); }
};

// Sums v over the lanes whose numbers differ in the bits D down to LAST, each lane
// keeping a part of the N sums (one at least), from the returned one on.
template <int N, int D, int LAST, int SIZE>
__device__ __forceinline__ int scatter_sums(float (&v)[SIZE]) {
  if constexpr (D < LAST) {
    return 0;
  } else if constexpr (N == 1) {
    v[0] += __shfl_xor(v[0], D);
    return scatter_sums<1, D / 2, LAST>(v);
  } else {
    const bool up = threadIdx.x & D;
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      const float send = up ? v[k] : v[k + N / 2], keep = up ? v[k + N / 2] : v[k];
      v[k] = keep + __shfl_xor(send, D);
    }
    return (up ? N / 2 : 0) + scatter_sums<N / 2, D / 2, LAST>(v);
  }
}

// The epilogue for one feature of R tokens.
template <int R, bool BACK, int FN>
__device__ __forceinline__ void finish_few(const LayerArgs &a, int64_t f, float (&h)[8]) {
  const int rows = static_cast<int>(a.rows);
  if constexpr (!BACK) {
    if (a.bias) {
      const float b = a.weight_f32 ? static_cast<const float *>(a.bias)[f] : to_f32(static_cast<const uint16_t *>(a.bias)[f]);
#pragma unroll
      for (int t = 0; t < R; ++t) h[t] = h[t] + b;
    }
    if (a.codes) {
      uint32_t top = 0;
#pragma unroll
      for (int t = 0; t < R; ++t)
        if (t < rows) top = max(top, __float_as_uint(h[t]) & 0x7fffffffu);
      const uint32_t s = a.fmt == kE4M3 ? act_scale<kE4M3>(top) : act_scale<kInt8>(top);
      float inv[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) inv[t] = a.fmt == kE4M3 ? act_inverse<kE4M3>(s) : act_inverse<kInt8>(s);
      const u32x2 w = a.fmt == kE4M3 ? encode8<kE4M3>(h, inv) : encode8<kInt8>(h, inv);
      a.scales[f] = static_cast<uint8_t>(s);
#pragma unroll
      for (int t = 0; t < R; ++t)
        if (t < rows) a.codes[t * a.pitch + f] = static_cast<uint8_t>(w[t >> 2] >> (8 * (t & 3)));
    }
    if constexpr (FN != kActNone) {
#pragma unroll
      for (int t = 0; t < R; ++t) h[t] = a.f32 ? act_value<FN, true>(h[t]) : short_value<FN>(h[t]);
    }
  } else if constexpr (FN != kActNone) {
    u32x2 w = {0, 0};
#pragma unroll
    for (int t = 0; t < R; ++t)
      if (t < rows) w[t >> 2] |= static_cast<uint32_t>(a.codes[t * a.pitch + f]) << (8 * (t & 3));
    float scale[8], x[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) scale[t] = act_scale_or_nan(a.scales[f]);
    if (a.fmt == kE4M3) decode8<kE4M3>(w, scale, x);
    else decode8<kInt8>(w, scale, x);
#pragma unroll
    for (int t = 0; t < R; ++t) h[t] = h[t] * (a.f32 ? act_slope<FN, true>(x[t]) : short_slope<FN>(x[t]));
  }
#pragma unroll
  for (int t = 0; t < R; ++t) {
    if (t < rows) {
      if (a.f32) {
        if (a.add) h[t] = h[t] + static_cast<const float *>(a.add)[t * a.ldadd + f];
        static_cast<float *>(a.y)[t * a.ldy + f] = h[t];
      } else {
        if (a.add) h[t] = h[t] + to_f32(static_cast<const uint16_t *>(a.add)[t * a.ldadd + f]);
        static_cast<uint16_t *>(a.y)[t * a.ldy + f] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(h[t]));
      }
    }
  }
}

// The activation as a constant: finish_few is small, the kernels in front of it are many.
template <int R, bool BACK>
__device__ __forceinline__ void finish_few(const LayerArgs &a, int64_t f, float (&h)[8]) {
  if (a.fn == kActGelu) finish_few<R, BACK, kActGelu>(a, f, h);
  else if (a.fn == kActGeluTanh) finish_few<R, BACK, kActGeluTanh>(a, f, h);
  else if (a.fn == kActSilu) finish_few<R, BACK, kActSilu>(a, f, h);
  else finish_few<R, BACK, kActNone>(a, f, h);
}

// Forward: a wavefront multiplies kFewRows rows of the weight with all tokens, 512
// steps of the contraction at a time.  SLICED: the four wavefronts of a workgroup
// share the rows and divide the contraction; otherwise each has rows of its own, which
// launch_layer takes where the contraction gives not every wavefront work.
template <int R, typename TW, typename TX, bool SLICED>
__global__ __launch_bounds__(kBlock) void layer_few_kernel(const LayerArgs a) {
  constexpr int FEATURES = SLICED ? kFewRows : kFewRows * kWaves;      // of a workgroup
  __shared__ float sums[kWaves][kFewRows * R];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t g0 = static_cast<int64_t>(blockIdx.x) * FEATURES, f0 = SLICED ? g0 : g0 + wave * kFewRows;
  const int64_t depth = a.shape.in;
  float acc[kFewRows * R];
#pragma unroll
  for (int k = 0; k < kFewRows * R; ++k) acc[k] = 0.0f;
  const TW *w0[kFewRows];
  const TX *x0[R];
#pragma unroll
  for (int o = 0; o < kFewRows; ++o) w0[o] = static_cast<const TW *>(a.weight) + min(f0 + o, a.features - 1) * depth + lane * 8;
#pragma unroll
  for (int t = 0; t < R; ++t) x0[t] = static_cast<const TX *>(a.x) + min(static_cast<int64_t>(t), a.rows - 1) * a.ldx + lane * 8;
  const auto add = [&](const Eight<TW> (&w)[kFewRows], const Eight<TX> (&x)[R]) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int o = 0; o < kFewRows; ++o)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[o * R + t] = __builtin_fmaf(w[o][k], x[t][k], acc[o * R + t]);
  };
  constexpr int STEP = SLICED ? 512 * kWaves : 512;
  int64_t k0 = SLICED ? wave * 512 : 0;
#pragma unroll 2
  for (; k0 + 512 <= depth; k0 += STEP) {
    Eight<TW> w[kFewRows];
    Eight<TX> x[R];
#pragma unroll
    for (int o = 0; o < kFewRows; ++o) w[o].load(w0[o] + k0);
#pragma unroll
    for (int t = 0; t < R; ++t) x[t].load(x0[t] + k0);
    add(w, x);
  }
  if (k0 < depth) {
    const int64_t n = depth - k0 - lane * 8;
    Eight<TW> w[kFewRows];
    Eight<TX> x[R];
#pragma unroll
    for (int o = 0; o < kFewRows; ++o) w[o].load_some(w0[o] + k0, n);
#pragma unroll
    for (int t = 0; t < R; ++t) x[t].load_some(x0[t] + k0, n);
    add(w, x);
  }
  const int at = scatter_sums<kFewRows * R, 32, 1>(acc);
  if ((lane & (64 / (kFewRows * R) - 1)) == 0) sums[wave][at] = acc[0];      // the lanes' last bits hold copies
  __syncthreads();
  const int c = threadIdx.x;
  if (c >= FEATURES || g0 + c >= a.features) return;
  float h[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    h[t] = 0.0f;
    if (t < R) {
      if constexpr (SLICED) {
#pragma unroll
        for (int s = 0; s < kWaves; ++s) h[t] += sums[s][c * R + t];
      } else {
        h[t] = sums[c / kFewRows][c % kFewRows * R + t];
      }
    }
  }
  finish_few<R, false>(a, g0 + c, h);
}

// Backward: kFewLanes lanes take eight features each of one row of the weight, the
// workgroup's 128 groups of them kFewEach rows each, all under way together: a slice
// of the contraction, whose sums go to `part` where there are several.  Neighbouring
// workgroups' features share cache lines, so they are given to one XCD.
template <int R, typename TW, typename TX>
__global__ __launch_bounds__(kFewBlock) void layer_few_back_kernel(const LayerArgs a, float *part) {
  constexpr int FEATURES = kFewLanes * 8, WAVES = kFewBlock / 64;
  __shared__ __attribute__((aligned(16))) float dys[kLayerSlice][R];
  __shared__ float sums[WAVES][R][FEATURES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = threadIdx.x / kFewLanes, l = threadIdx.x % kFewLanes;
  const uint32_t xcd = blockIdx.x % kXcds, place = xcd * (gridDim.x / kXcds) + min(xcd, gridDim.x % kXcds) + blockIdx.x / kXcds;
  const int64_t g0 = static_cast<int64_t>(place) * FEATURES, f = g0 + l * 8, c0 = static_cast<int64_t>(blockIdx.y) * kLayerSlice;
  const int rows = static_cast<int>(min(static_cast<int64_t>(kLayerSlice), a.shape.out - c0));
  const int64_t n = a.features - f;
  Eight<TW> w[kFewEach];
#pragma unroll
  for (int e = 0; e < kFewEach; ++e) {
    const TW *p = static_cast<const TW *>(a.weight) + (c0 + min(group + e * kFewGroups, rows - 1)) * a.features + f;
    if (n >= 8) w[e].load(p);
    else w[e].load_some(p, n);
  }
#pragma unroll
  for (int t = 0; t < R; ++t)
    for (int o = threadIdx.x; o < rows; o += kFewBlock)
      dys[o][t] = t < a.rows ? to_f32(static_cast<const TX *>(a.x)[t * a.ldx + c0 + o]) : 0.0f;
  __syncthreads();
  float acc[R * 8];
#pragma unroll
  for (int k = 0; k < R * 8; ++k) acc[k] = 0.0f;
#pragma unroll
  for (int e = 0; e < kFewEach; ++e) {
    const int o = group + e * kFewGroups;
    if (o < rows) {
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const float y = dys[o][t];
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[t * 8 + k] = __builtin_fmaf(y, w[e][k], acc[t * 8 + k]);
      }
    }
  }
  constexpr int KEPT = R * 8 * kFewLanes / 64 > 0 ? R * 8 * kFewLanes / 64 : 1;      // sums that a lane is left with
  const int at = scatter_sums<R * 8, 32, kFewLanes>(acc);
  // with fewer sums than lanes the last of the lanes' bits hold copies
  if (R * 8 * kFewLanes >= 64 || (lane & kFewLanes) == 0) {
#pragma unroll
    for (int k = 0; k < KEPT; ++k) sums[wave][(at + k) / 8][l * 8 + (at + k) % 8] = acc[k];
  }
  __syncthreads();
  const int c = threadIdx.x;
  if (c >= FEATURES || g0 + c >= a.features) return;
  float h[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    h[t] = 0.0f;
    if (t < R) {
#pragma unroll
      for (int s = 0; s < WAVES; ++s) h[t] += sums[s][t][c];
    }
  }
  if (part) {
    const int64_t ldp = (a.features + 3) / 4 * 4;
#pragma unroll
    for (int t = 0; t < R; ++t)
      if (t < a.rows) part[(blockIdx.y * a.rows + t) * ldp + g0 + c] = h[t];
    return;
  }
  finish_few<R, true>(a, g0 + c, h);
}

// ---------------------------------------------------------------------------
// operands that the product cannot read as they are
// ---------------------------------------------------------------------------
// A matrix [rows][cols] as bf16 parts [PARTS][rows][pitch], pitch a multiple of 64
// and its end zero: fp32 as three parts, bf16 whose rows do not start on 16 bytes
// as one.
struct PackArgs {
  const void *from;
  bool f32;
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
__device__ __forceinline__ void pack_units(const PackArgs &a, int64_t first, int64_t step) {
  const int64_t units = a.pitch / 8, total = a.rows * units;
  for (int64_t id = first; id < total; id += step) {
    const int64_t r = id / units, c = (id - r * units) * 8;
    Eight<T> v;
    const T *p = static_cast<const T *>(a.from) + r * a.ld + c;
    if (c + 8 <= a.cols) v.load(p);
    else v.load_some(p, a.cols - c);
    uint16_t *out = a.to + r * a.pitch + c;
    if constexpr (sizeof(T) == 2) {
      __builtin_memcpy(__builtin_assume_aligned(out, 16), v.v, 16);
    } else {
      uint16_t w[3][8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint16_t h[3];
        parts3(v.v[k], h);
#pragma unroll
        for (int s = 0; s < 3; ++s) w[s][k] = h[s];
      }
#pragma unroll
      for (int s = 0; s < 3; ++s) __builtin_memcpy(__builtin_assume_aligned(out + s * a.rows * a.pitch, 16), w[s], 16);
    }
  }
}

// The weight by the first `blocks` workgroups, x or dy by the others.
__global__ __launch_bounds__(kBlock) void pack_kernel(const PackArgs a, const PackArgs b, uint32_t blocks) {
  const bool first = blockIdx.x < blocks;
  const PackArgs &p = first ? a : b;
  const int64_t at = static_cast<int64_t>(first ? blockIdx.x : blockIdx.x - blocks) * kBlock + threadIdx.x;
  const int64_t step = static_cast<int64_t>(first ? blocks : gridDim.x - blocks) * kBlock;
  if (p.f32) pack_units<float>(p, at, step);
  else pack_units<uint16_t>(p, at, step);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Calls f with the direction and the activation as constants.
template <typename F>
void by_kind(const LayerArgs &a, F &&f) {
  const auto by_fn = [&](auto back) {
    if (a.fn == kActGelu) f(back, std::integral_constant<int, kActGelu>{});
    else if (a.fn == kActGeluTanh) f(back, std::integral_constant<int, kActGeluTanh>{});
    else if (a.fn == kActSilu) f(back, std::integral_constant<int, kActSilu>{});
    else f(back, std::integral_constant<int, kActNone>{});
  };
  if (a.shape.back) by_fn(std::true_type{});
  else by_fn(std::false_type{});
}

template <int BF, int BT, int WF, int WT, int KT, int PA, int PB, bool RAW, int STAGES, int WGS>
void layer_one(const LayerArgs &a, const LayerPlan &p, const Product &q, float *part, hipStream_t s) {
  const Split sp{p.m_tiles, p.n_tiles, p.splits, p.turns_each};
  const dim3 grid(static_cast<unsigned>(p.m_tiles) * p.n_tiles * p.splits);
  by_kind(a, [&](auto back, auto fn) {
    layer_kernel<BF, BT, WF, WT, KT, PA, PB, RAW, STAGES, WGS, decltype(back)::value, decltype(fn)::value>
        <<<grid, 64 * WF * WT, 0, s>>>(a, q, sp, part);
  });
}

template <int R, typename TW, typename TX>
void layer_few(const LayerArgs &a, int slices, float *part, hipStream_t s) {
  const auto groups = [&](int64_t each) { return static_cast<unsigned>((a.features + each - 1) / each); };
  // Wavefronts that share their rows, but where four times 512 steps are more than there are:
  // 8 tokens of 1024 -> 8192 in bf16 15.4 us so and 7.5 the other way, of 2048 -> 8192 17.9
  // and 9.6; of 8192 -> 2048 10.5 and 19.1, one token of 8192 -> 8192 20.6 and 28.7.
  if (a.shape.back) {
    layer_few_back_kernel<R, TW, TX><<<dim3(groups(kFewLanes * 8), slices), kFewBlock, 0, s>>>(a, part);
    return;
  }
  if constexpr (R > 1) {
    if (a.shape.in <= 512 * kWaves && a.features >= 4096) {
      layer_few_kernel<R, TW, TX, false><<<groups(kFewRows * kWaves), kBlock, 0, s>>>(a);
      return;
    }
  }
  layer_few_kernel<R, TW, TX, true><<<groups(kFewRows), kBlock, 0, s>>>(a);
}

template <typename TW, typename TX>
void layer_few_by_rows(const LayerArgs &a, int slices, float *part, hipStream_t s) {
  if (a.rows == 1) layer_few<1, TW, TX>(a, slices, part, s);
  else if (a.rows <= 4) layer_few<4, TW, TX>(a, slices, part, s);
  else layer_few<8, TW, TX>(a, slices, part, s);
}

char *work_at(const LayerArgs &a, size_t bytes) { return static_cast<char *>(a.work) + bytes; }

}  // namespace

void launch_layer_pack(const LayerArgs &a, const LayerPlan &p, hipStream_t s) {
  const int64_t depth = layer_depth(a.shape);
  const PackArgs w{a.weight, a.weight_f32, a.shape.in, static_cast<uint16_t *>(a.work), a.shape.out, a.shape.in, layer_pitch(a.shape.in)};
  const PackArgs x{a.x, a.f32, a.ldx, reinterpret_cast<uint16_t *>(work_at(a, p.a_bytes)), a.rows, depth, layer_pitch(depth)};
  const auto blocks = [](const PackArgs &q) {
    return static_cast<uint32_t>(std::min<int64_t>((q.rows * (q.pitch / 8) + kBlock - 1) / kBlock, 1 << 15));
  };
  const uint32_t first = p.pack_a ? blocks(w) : 0, others = p.pack_b ? blocks(x) : 0;
  pack_kernel<<<first + others, kBlock, 0, s>>>(w, x, first);
}

void launch_layer(const LayerArgs &a, const LayerPlan &p, hipStream_t s) {
  float *part = p.splits > 1 ? reinterpret_cast<float *>(work_at(a, p.a_bytes + p.b_bytes)) : nullptr;
  if (p.tile < 0) {
    if (a.weight_f32) {
      if (a.f32) layer_few_by_rows<float, float>(a, p.splits, part, s);
      else layer_few_by_rows<float, uint16_t>(a, p.splits, part, s);
    } else {
      if (a.f32) layer_few_by_rows<uint16_t, float>(a, p.splits, part, s);
      else layer_few_by_rows<uint16_t, uint16_t>(a, p.splits, part, s);
    }
    return;
  }
  const int64_t depth = layer_depth(a.shape);
  Product q{};
  q.rows = a.rows;
  q.features = a.features;
  q.depth = depth % 8 == 0 ? depth : layer_pitch(depth);      // then operands that lie along k are packed (or fp32 as they lie)
  q.true_depth = depth;
  q.a = p.pack_a ? a.work : a.weight;
  q.lda = p.pack_a ? layer_pitch(a.shape.in) : a.shape.in;
  q.a_part = a.shape.out * q.lda;
  q.b = p.pack_b ? work_at(a, p.a_bytes) : a.x;
  q.ldb = p.pack_b ? layer_pitch(depth) : a.ldx;
  q.b_part = a.rows * q.ldb;
  if (p.a_parts * p.b_parts == 1) {
    if (p.tile == 0) layer_one<256, 256, 4, 2, 64, 1, 1, false, 2, 1>(a, p, q, part, s);
    else if (p.tile == 1) layer_one<128, 128, 4, 2, 64, 1, 1, false, 2, 2>(a, p, q, part, s);
    else layer_one<128, 32, 4, 1, 64, 1, 1, false, 4, 2>(a, p, q, part, s);
  } else if (p.a_parts == 3 && p.b_parts == 3) {
    if (p.tile == 0) layer_one<128, 128, 2, 2, 32, 3, 3, false, 3, 1>(a, p, q, part, s);
    else if (p.tile == 1) layer_one<128, 64, 4, 1, 32, 3, 3, false, 4, 1>(a, p, q, part, s);
    else layer_one<128, 64, 4, 1, 32, 3, 3, true, 2, 1>(a, p, q, part, s);
  } else if (p.a_parts == 3) {
    if (p.tile == 0) layer_one<128, 128, 2, 2, 32, 3, 1, false, 2, 2>(a, p, q, part, s);
    else if (p.tile == 1) layer_one<128, 64, 4, 1, 32, 3, 1, false, 2, 2>(a, p, q, part, s);
    else layer_one<128, 64, 4, 1, 32, 3, 1, true, 2, 1>(a, p, q, part, s);
  } else {
    if (p.tile == 0) layer_one<128, 128, 2, 2, 32, 1, 3, false, 2, 2>(a, p, q, part, s);
    else if (p.tile == 1) layer_one<128, 64, 4, 1, 32, 1, 3, false, 2, 2>(a, p, q, part, s);
    else layer_one<128, 64, 4, 1, 32, 1, 3, true, 2, 1>(a, p, q, part, s);
  }
}

void launch_layer_join(const LayerArgs &a, const LayerPlan &p, hipStream_t s) {
  const float *part = reinterpret_cast<const float *>(work_at(a, p.a_bytes + p.b_bytes));
  const dim3 grid(static_cast<unsigned>((a.rows + 31) / 32 * ((a.features + kJoinWidth - 1) / kJoinWidth)));
  by_kind(a, [&](auto back, auto fn) {
    layer_join_kernel<decltype(back)::value, decltype(fn)::value><<<grid, kBlock, 0, s>>>(a, part, p.splits);
  });
}

}  // namespace ob
