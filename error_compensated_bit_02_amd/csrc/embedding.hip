// Embedding lookup with scaling, and its gradient by sorted tokens (gfx950).
//
//   lookup    out[t] = scale * table[id_t]
//   gradient  dE[v] = scale * sum over t with id_t = v, ascending t, of dy[t]
//
// An id below 0 is padding: a zero row, no gradient.  An id at or past the
// table's end gives a NaN row in the lookup, where it shows, and no gradient;
// no access ever depends on an unchecked id.
//
// Gradient.  Tokens are ordered by (id, t) and summed run by run: no atomic
// touches a sum, so results repeat bit for bit.
//  1. order: each workgroup sorts one tile of kSortTile tokens by id in LDS,
//     four bits a pass (stable, so equal ids stay in token order);
//  2. merge: kMergeWays sorted runs become one; an element's place is its
//     index in its own run plus its rank in each other run, found by binary
//     search;
//  3. sum: one wavefront sums a chunk of consecutive sorted tokens of one
//     slice of columns in fp32; a run of equal ids inside the chunk is
//     written out, the parts of a run that crosses chunks go to the workspace.
//     dY is read once, by loads that bypass the caches (kept in them it
//     pushed out the gradient's lines: 58 us for 32768 x 2048, 35 without);
//  4. join: the chunk where such a run begins adds its parts in order.
// A gradient that is not accumulated is written whole, rows without a token as
// zeros: further workgroups of the order launch zero all of it while it sorts
// (a sort alone takes 13 us, the gradient of 50257 x 2048 in bf16 28 us).
// Rows that have a token are then written twice; finding those that have none
// and zeroing only them, beside the sums, was slower: 97 us against 94 for
// 32768 tokens into that gradient, 44 against 35 for 4096 into 30522 x 1024.
// Up to kFewTokens tokens are summed without steps 1, 2 and 4, behind a launch
// that only zeroes (few_kernel).
#include "internal.h"

#include <algorithm>

#pragma clang fp contract(off)

namespace ob {
namespace {

constexpr int kSortTile = 4096;
constexpr int kSortThreads = 1024;
constexpr int kSortShift = 12;          // log2(kSortTile)
constexpr int kMergeWays = 8;
constexpr int kLeastChunk = 8;          // sorted tokens summed by one wavefront, at least
constexpr uint32_t kNoId = 0xffffffffu; // sorts last, never summed
constexpr int kFewTokens = 128;         // up to here without sorting (few_kernel)
constexpr int kFewEach = 16;            // of them a wavefront's own
constexpr int kFewThreads = kFewTokens / kFewEach * 64;

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  bf16x2 r;
  r[0] = static_cast<__bf16>(a);
  r[1] = static_cast<__bf16>(b);
  return __builtin_bit_cast(uint32_t, r);
}

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

// N consecutive elements as fp32 and back: 16-byte accesses where N > 1 (the
// caller has checked alignment).  read_once: loads that leave the caches to
// others.
template <typename T, int N>
struct Vec {
  static __device__ __forceinline__ void read_once(const T *p, float (&v)[N]) {
    if constexpr (N == 1) {
      const T x = __builtin_nontemporal_load(p);
      if constexpr (sizeof(T) == 4) v[0] = x;
      else v[0] = __uint_as_float(static_cast<uint32_t>(x) << 16);
    } else {
      constexpr int kEach = 16 / sizeof(T);
#pragma unroll
      for (int k = 0; k < N; k += kEach) {
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
    }
  }
  static __device__ __forceinline__ void load(const T *p, float (&v)[N]) {
    if constexpr (N == 1) {
      if constexpr (sizeof(T) == 4) v[0] = *p;
      else v[0] = __uint_as_float(static_cast<uint32_t>(*p) << 16);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p + k);
        v[k] = a.x, v[k + 1] = a.y, v[k + 2] = a.z, v[k + 3] = a.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; k += 8) {
        const uint4 a = *reinterpret_cast<const uint4 *>(p + k);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          v[k + 2 * h] = __uint_as_float(w[h] << 16);
          v[k + 2 * h + 1] = __uint_as_float(w[h] & 0xffff0000u);
        }
      }
    }
  }
  static __device__ __forceinline__ void store(T *p, const float (&v)[N]) {
    if constexpr (N == 1) {
      if constexpr (sizeof(T) == 4) *p = v[0];
      else *p = static_cast<uint16_t>(pack_bf16(v[0], 0.0f));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < N; k += 4) *reinterpret_cast<float4 *>(p + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
    } else {
#pragma unroll
      for (int k = 0; k < N; k += 8)
        *reinterpret_cast<uint4 *>(p + k) = make_uint4(pack_bf16(v[k], v[k + 1]), pack_bf16(v[k + 2], v[k + 3]),
                                                       pack_bf16(v[k + 4], v[k + 5]), pack_bf16(v[k + 6], v[k + 7]));
    }
  }
};

__device__ __forceinline__ int64_t id_at(const EmbedArgs &a, int64_t t) {
  return a.ids64 ? static_cast<const int64_t *>(a.ids)[t]
                 : static_cast<int64_t>(static_cast<const int32_t *>(a.ids)[t]);
}

// ---------------------------------------------------------------------------
// lookup: `lanes` threads a row, N columns a thread and turn
// ---------------------------------------------------------------------------
template <typename T, int N>
__global__ __launch_bounds__(kBlock) void lookup_kernel(const EmbedArgs a, int lanes_log2) {
  const int lanes = 1 << lanes_log2;
  const int64_t t = (static_cast<int64_t>(blockIdx.x) << (8 - lanes_log2)) + (threadIdx.x >> lanes_log2);
  if (t >= a.tokens) return;
  const int64_t id = id_at(a, t);
  const bool inside = id >= 0 && id < a.vocab;
  const float *row = a.table + (inside ? id : 0) * a.dim;
  T *out = static_cast<T *>(a.out) + t * a.ldo;
  for (int64_t c = static_cast<int64_t>(threadIdx.x & (lanes - 1)) * N; c < a.dim; c += lanes * N) {
    float v[N];
    if (inside) {
      Vec<float, N>::load(row + c, v);
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] *= a.scale;
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = id < 0 ? 0.0f : __uint_as_float(0x7fc00000u);
    }
    Vec<T, N>::store(out + c, v);
  }
}

// ---------------------------------------------------------------------------
// order
// ---------------------------------------------------------------------------
struct Order {
  uint32_t *key[2];      // ids in sorted order, kNoId for those without a row
  uint32_t *pos[2];      // their tokens
  float *part;           // [chunks][2][dim] parts of runs that cross chunks
  int chunk;             // sorted tokens of a chunk
  int64_t chunks;
  int passes;            // merge passes; the result is in key/pos[passes & 1]
};

// Sorted tokens a wavefront sums.  More of them mean fewer parts to join,
// fewer of them more wavefronts: the most that still leaves a few thousand.
int chunk_of(int64_t tokens, int64_t dim) {
  const int64_t slices = (dim + 511) / 512;
  int chunk = 32;
  while (chunk > kLeastChunk && tokens * slices / chunk < 4096) chunk /= 2;
  return chunk;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

Order order_of(const EmbedArgs &a) {
  Order o{};
  unsigned char *p = static_cast<unsigned char *>(a.work);
  const size_t b = up256(static_cast<size_t>(a.tokens) * 4);
  o.passes = 0;
  for (int64_t run = kSortTile; run < a.tokens; run *= kMergeWays) ++o.passes;
  const int sides = o.passes ? 2 : 1;
  for (int k = 0; k < sides; ++k) {
    o.key[k] = reinterpret_cast<uint32_t *>(p);
    o.pos[k] = reinterpret_cast<uint32_t *>(p + b);
    p += 2 * b;
  }
  o.part = reinterpret_cast<float *>(p);
  o.chunk = chunk_of(a.tokens, a.dim);
  o.chunks = (a.tokens + o.chunk - 1) / o.chunk;
  return o;
}

// Inclusive sum over the lanes of a wavefront: within rows of 16 lanes, then
// across the rows.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t shifted(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += shifted<0x111, 0xf>(v);   // from 1, 2, 4 and 8 lanes below in the row
  v += shifted<0x112, 0xf>(v);
  v += shifted<0x114, 0xf>(v);
  v += shifted<0x118, 0xf>(v);
  v += shifted<0x142, 0xa>(v);   // the last lane of a row to the next, rows 1 and 3
  v += shifted<0x143, 0xc>(v);   // lane 31 to rows 2 and 3
  return v;
}

// K: uint32_t while an id and a place in the tile fit in 32 bits, else uint64_t.
// `bits`: of an id, the one behind the table's last included.
template <typename K>
__global__ __launch_bounds__(kSortThreads) void order_kernel(const EmbedArgs a, uint32_t *key, uint32_t *pos, int bits,
                                                             int sort_blocks, int64_t zero_bytes) {
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) >= sort_blocks) {   // zero the gradient
    const int64_t n = zero_bytes / 16;
    uint4 *g = static_cast<uint4 *>(a.grad);
    const int64_t step = static_cast<int64_t>(gridDim.x - sort_blocks) * kSortThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x - sort_blocks) * kSortThreads + tid;
    for (int64_t i = first; i < n; i += step) g[i] = make_uint4(0, 0, 0, 0);
    // the last bytes of a gradient that ends inside 16 bytes, two at a time (padding stays untouched)
    if (first < (zero_bytes - n * 16) / 2) reinterpret_cast<uint16_t *>(g + n)[first] = 0;
    return;
  }
  // Element e = j * kSortThreads + tid.  A group is the 64 elements of one j
  // and wavefront; group j * kSortWaves + wave holds the e's in order.  A
  // pass counts each digit in each group, scans the counts digit by digit and
  // group by group, and moves every element to its digit's and group's start
  // plus its rank among the group's equals.  Two sets of counts: while one is
  // in use the other is cleared.
  constexpr int kPer = kSortTile / kSortThreads, kSortWaves = kSortThreads / 64, kGroups = kPer * kSortWaves;
  static_assert(kGroups == 64 && 16 * kGroups == kSortThreads, "one count a thread, one digit a wavefront");
  __shared__ K s[kSortTile];
  __shared__ uint32_t counts[2][16 * kGroups], total[16];
  const int lane = tid & 63, wave = tid >> 6;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortTile;
  const int len = static_cast<int>(min(static_cast<int64_t>(kSortTile), a.tokens - base));
  const int per = (len + kSortThreads - 1) / kSortThreads;    // j's in use
  const K none = static_cast<K>(a.vocab);   // the id behind the table's last; also of elements past the end, which stay behind
  K k[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = j * kSortThreads + tid;
    K id = none;
    if (e < len) {
      const int64_t v = id_at(a, base + e);
      if (v >= 0 && v < a.vocab) id = static_cast<K>(v);
    }
    k[j] = (id << kSortShift) | static_cast<K>(e);
  }
  counts[0][tid] = 0;
  __syncthreads();
  for (int shift = kSortShift, side = 0; shift < kSortShift + bits; shift += 4, side ^= 1) {
    uint32_t *const count = counts[side];
    counts[side ^ 1][tid] = 0;
    uint32_t rank[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (j < per) {
        const uint32_t digit = static_cast<uint32_t>(k[j] >> shift) & 15u;
        uint32_t same_lo = ~0u, same_hi = ~0u;    // lanes with the same digit
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t bit = __builtin_amdgcn_sbfe(digit, b, 1);   // all ones or zeros
          const uint64_t set = __ballot(bit != 0);
          same_lo &= ~(static_cast<uint32_t>(set) ^ bit);
          same_hi &= ~(static_cast<uint32_t>(set >> 32) ^ bit);
        }
        rank[j] = __builtin_amdgcn_mbcnt_hi(same_hi, __builtin_amdgcn_mbcnt_lo(same_lo, 0));
        if (rank[j] == 0)
          count[digit * kGroups + j * kSortWaves + wave] = static_cast<uint32_t>(__popc(same_lo) + __popc(same_hi));
      }
    }
    __syncthreads();
    const uint32_t mine = count[tid];        // digit `wave`, group `lane`
    const uint32_t upto = wave_scan(mine);
    if (lane == 63) total[wave] = upto;
    __syncthreads();
    uint32_t start = upto - mine;
#pragma unroll
    for (int w = 0; w < 16; ++w)
      if (w < wave) start += total[w];
    count[tid] = start;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (j < per) {
        const uint32_t digit = static_cast<uint32_t>(k[j] >> shift) & 15u;
        s[count[digit * kGroups + j * kSortWaves + wave] + rank[j]] = k[j];
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j < per) k[j] = s[j * kSortThreads + tid];
    // the next pass writes s only behind its barriers
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = j * kSortThreads + tid;
    if (e < len) {
      const K id = k[j] >> kSortShift;
      key[base + e] = id == none ? kNoId : static_cast<uint32_t>(id);
      pos[base + e] = static_cast<uint32_t>(base) + static_cast<uint32_t>(k[j] & (kSortTile - 1));
    }
  }
}

// Merges kMergeWays sorted runs of `run` elements each.  Searching in memory
// (L2) took 9 us for 32768 tokens, with the group's keys put into LDS first 16.
__global__ __launch_bounds__(kBlock) void merge_kernel(const uint32_t *key, const uint32_t *pos, uint32_t *key_out,
                                                       uint32_t *pos_out, int64_t tokens, int64_t run) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  // runs and groups hold whole workgroups of elements
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * kBlock / run, first = mine / kMergeWays * kMergeWays;
  const int64_t group = first * run;
  const uint32_t *from = key + group;
  if (j >= tokens) return;
  const uint32_t k = key[j];
  int64_t place = j - (mine - first) * run;
  uint32_t top = 1;                        // smallest power of two past the run's length
  while (top <= run) top *= 2;
  uint32_t start[kMergeWays], len[kMergeWays], below[kMergeWays];
#pragma unroll
  for (int u = 0; u < kMergeWays; ++u) {
    const int64_t left = tokens - group - u * run;
    len[u] = first + u == mine || left <= 0 ? 0u : static_cast<uint32_t>(min(left, run));
    start[u] = len[u] ? static_cast<uint32_t>(u * run) : 0u;
    below[u] = 0;                          // elements known to come before (k, this run)
  }
  // every probe reads, inside its run (or the group's first key), so that the
  // searches' reads overlap
  for (uint32_t step = top / 2; step > 0; step /= 2) {
    uint32_t other[kMergeWays];
#pragma unroll
    for (int u = 0; u < kMergeWays; ++u) other[u] = from[start[u] + max(min(below[u] + step, len[u]), 1u) - 1];
#pragma unroll
    for (int u = 0; u < kMergeWays; ++u) {
      const uint32_t probe = below[u] + step;
      const bool before = first + u < mine ? other[u] <= k : other[u] < k;
      below[u] = probe <= len[u] && before ? probe : below[u];
    }
  }
#pragma unroll
  for (int u = 0; u < kMergeWays; ++u) place += below[u];
  key_out[place] = k;
  pos_out[place] = pos[j];
}

// ---------------------------------------------------------------------------
// sum and join
// ---------------------------------------------------------------------------
template <typename G, int N>
__device__ __forceinline__ void write_row(const EmbedArgs &a, uint32_t id, int64_t c, const float (&sum)[N]) {
  G *p = static_cast<G *>(a.grad) + static_cast<int64_t>(id) * a.dim + c;
  float v[N];
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = sum[k] * a.scale;
  if (a.accumulate) {
    float old[N];
    Vec<G, N>::load(p, old);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += old[k];
  }
  Vec<G, N>::store(p, v);
}

template <typename T, typename G, int N>
__global__ __launch_bounds__(kBlock) void sum_kernel(const EmbedArgs a, const uint32_t *key, const uint32_t *pos,
                                                     float *part, int run, int64_t chunks, int slices) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= chunks * slices) return;
  const int64_t chunk = unit / slices;
  const int64_t c = (static_cast<int64_t>(unit - chunk * slices) * 64 + lane) * N;
  const bool live = c < a.dim;
  const int64_t j0 = chunk * run;
  const int len = static_cast<int>(min(static_cast<int64_t>(run), a.tokens - j0));
  uint32_t lk = kNoId, lp = 0;
  if (lane < len) {
    lk = key[j0 + lane];
    lp = pos[j0 + lane];
  }
  const uint32_t before = j0 > 0 ? key[j0 - 1] : kNoId;
  const uint32_t after = j0 + len < a.tokens ? key[j0 + len] : kNoId;
  float sum[N];
#pragma unroll
  for (int k = 0; k < N; ++k) sum[k] = 0.0f;
  bool head = true;                        // the run at hand is the chunk's first
  const T *dy = static_cast<const T *>(a.dy) + (live ? c : 0);
  for (int b = 0; b < len; b += 8) {
    float v[8][N];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t p = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(lp), (b + u) & 31));
      Vec<T, N>::read_once(dy + static_cast<int64_t>(p) * a.lddy, v[u]);   // absent tokens read token 0, unused
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = b + u;
      if (j >= len) break;
      const uint32_t k = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(lk), j));
      if (k == kNoId) return;              // all that follow are without a row
#pragma unroll
      for (int x = 0; x < N; ++x) sum[x] += v[u][x];
      const bool last = j + 1 == len;
      const uint32_t next = last ? after : static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(lk), j + 1));
      if (last || next != k) {
        const bool from_before = head && before == k;
        const bool goes_on = last && next == k;
        if (live) {
          if (from_before || goes_on) Vec<float, N>::store(part + (chunk * 2 + (from_before ? 0 : 1)) * a.dim + c, sum);
          else write_row<G, N>(a, k, c, sum);
        }
#pragma unroll
        for (int x = 0; x < N; ++x) sum[x] = 0.0f;
        head = false;
      }
    }
  }
}

// One workgroup per (chunk, slice); it has work where a run begins in the
// chunk and goes on past its end.  The run's parts are split into kWaves
// consecutive ranges, and the ranges' sums added in order.
template <typename G, int N>
__global__ __launch_bounds__(kBlock) void join_kernel(const EmbedArgs a, const uint32_t *key, const float *part,
                                                      int run, int slices) {
  const int64_t chunk = blockIdx.x / slices;
  const int64_t j0 = chunk * run, j1 = j0 + run;
  if (j1 >= a.tokens) return;
  const uint32_t k = key[j1 - 1];
  if (k == kNoId || key[j1] != k) return;
  if (key[j0] == k && j0 > 0 && key[j0 - 1] == k) return;    // began earlier
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (static_cast<int64_t>(blockIdx.x - chunk * slices) * 64 + lane) * N;
  const bool live = c < a.dim;
  // later chunks that hold a part: those that begin with the run's id, 64 at a look
  int64_t parts = 0;
  for (;;) {
    const int64_t j = j1 + (parts + lane) * run;
    const uint64_t same = __ballot(j < a.tokens && key[j] == k);
    parts += __popcll(same);
    if (~same) break;
  }
  const int64_t each = (parts + kWaves - 1) / kWaves;
  const int64_t p0 = min(parts, wave * each), p1 = min(parts, p0 + each);
  const float *src = part + (chunk + 1) * 2 * a.dim + (live ? c : 0);
  float sum[N];
#pragma unroll
  for (int x = 0; x < N; ++x) sum[x] = 0.0f;
#pragma unroll 8
  for (int64_t p = p0; p < p1; ++p) {
    float v[N];
    Vec<float, N>::load(src + p * 2 * a.dim, v);
#pragma unroll
    for (int x = 0; x < N; ++x) sum[x] += v[x];
  }
  __shared__ float s[kWaves][64 * N];
#pragma unroll
  for (int x = 0; x < N; ++x) s[wave][lane * N + x] = sum[x];
  __syncthreads();
  if (wave != 0 || !live) return;
  Vec<float, N>::load(part + (chunk * 2 + 1) * a.dim + c, sum);
  for (int w = 0; w < kWaves; ++w) {
#pragma unroll
    for (int x = 0; x < N; ++x) sum[x] += s[w][lane * N + x];
  }
  write_row<G, N>(a, k, c, sum);
}

// A few tokens, unsorted: a workgroup takes one token and slice of columns.
// Comparisons and ballots tell which tokens share its id; if it is their
// first, each wavefront sums those among 16 tokens of its own, in order, and
// the wavefronts' sums are added in order.  Bound by the latency of ids, rows
// and, in one place, of the rows that a wavefront reads one batch after the
// other.  Against the sort, whole gradient of 30522 x 768 in fp32 (its zeroing
// takes 14 us): 77 different tokens 16.6 us against 20.9, 77 times the same
// 21.7 against 21.9, 128 times the same 25.0 against 22.4; accumulated 8.7
// against 14.6 either way.  With up to 256 tokens the same one 256 times takes
// 34 us against 23, and at 8192 columns different ones 45 against 19.
template <typename T, typename G, int N>
__global__ __launch_bounds__(kFewThreads) void few_kernel(const EmbedArgs a, int slices) {
  constexpr int kFewWaves = kFewThreads / 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = static_cast<int>(blockIdx.x);
  const int64_t row = id_at(a, t);
  uint32_t same[kFewWaves];                // bit b of word w: token kFewEach * w + b
#pragma unroll
  for (int s = 0; s < kFewTokens / 64; ++s) {
    const int other = s * 64 + lane;
    const uint64_t set = __ballot(other < a.tokens && id_at(a, other < a.tokens ? other : 0) == row);
#pragma unroll
    for (int w = 0; w < 64 / kFewEach; ++w)
      same[s * (64 / kFewEach) + w] = static_cast<uint32_t>(set >> (w * kFewEach)) & ((1u << kFewEach) - 1);
  }
  if (row < 0 || row >= a.vocab) return;
  uint32_t earlier = 0, mine = 0;
  bool alone = true;                       // all of the row's tokens belong to this token's wavefront
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w) {
    if (w < t / kFewEach) earlier |= same[w];
    if (w == t / kFewEach) earlier |= same[w] & ((1u << (t % kFewEach)) - 1);
    else alone = alone && same[w] == 0;
    if (w == wave) mine = same[w];
  }
  if (earlier) return;                     // the earliest sums
  if (alone && wave != t / kFewEach) return;
  __shared__ float parts[kFewWaves][64 * N];
  for (int slice = blockIdx.y; slice < slices; slice += gridDim.y) {
    const int64_t c = (static_cast<int64_t>(slice) * 64 + lane) * N;
    const bool live = c < a.dim;
    const T *dy = static_cast<const T *>(a.dy) + (live ? c : 0) + static_cast<int64_t>(wave) * kFewEach * a.lddy;
    float sum[N];
#pragma unroll
    for (int k = 0; k < N; ++k) sum[k] = 0.0f;
    uint32_t left = mine;
    int at = 0;
    while (left) {
      const int n = __popc(left);
      float v[8][N];
#pragma unroll
      for (int u = 0; u < 8; ++u) {        // reads past the last are of the last again, unused
        if (left) at = __builtin_ctz(left);
        left &= left - 1;
        Vec<T, N>::read_once(dy + at * a.lddy, v[u]);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (u < n) {
#pragma unroll
          for (int k = 0; k < N; ++k) sum[k] += v[u][k];
        }
      }
    }
    if (!alone) {
      __syncthreads();                     // the last slice's parts have been read
#pragma unroll
      for (int k = 0; k < N; ++k) parts[wave][k * 64 + lane] = sum[k];
      __syncthreads();
      if (wave != 0) continue;
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) {
#pragma unroll
        for (int k = 0; k < N; ++k) sum[k] += parts[w][k * 64 + lane];
      }
    }
    if (live) write_row<G, N>(a, static_cast<uint32_t>(row), c, sum);
  }
}

template <typename T, typename G, int N>
void sum_one(const EmbedArgs &a, hipStream_t s) {
  const int slices = static_cast<int>((a.dim + 64 * N - 1) / (64 * N));
  if (embed_few(a)) {
    few_kernel<T, G, N><<<dim3(a.tokens, std::min(slices, 1024)), kFewThreads, 0, s>>>(a, slices);
    return;
  }
  const Order o = order_of(a);
  const int side = o.passes & 1;
  const int64_t units = o.chunks * slices;
  sum_kernel<T, G, N><<<dim3((units + kWaves - 1) / kWaves), kBlock, 0, s>>>(a, o.key[side], o.pos[side], o.part, o.chunk,
                                                                             o.chunks, slices);
  if (o.chunks > 1) join_kernel<G, N><<<dim3(units), kBlock, 0, s>>>(a, o.key[side], o.part, o.chunk, slices);
}

template <typename T, typename G>
void sum_by_width(const EmbedArgs &a, hipStream_t s) {
  // eight columns a lane where every row of dy and of the gradient starts on 16 bytes
  if (a.dim % 8 == 0 && a.lddy % 8 == 0 && reinterpret_cast<uintptr_t>(a.dy) % 16 == 0) sum_one<T, G, 8>(a, s);
  else sum_one<T, G, 1>(a, s);
}

}  // namespace

bool lookup_fits(int64_t tokens) { return tokens <= kMaxGrid; }   // a workgroup a token at most

bool embed_grad_fits(int64_t tokens, int64_t vocab, int64_t dim) {
  // Sorted ids are 32-bit, the largest standing for none; the join has a workgroup per chunk and slice, which is
  // 64 columns wide where rows are not vectors.  Chunks are shorter than 32 tokens only where tokens times slices
  // of 512 columns stay below 2^17 (chunk_of), and those make far fewer workgroups than the limit.
  return tokens <= kMaxGrid && vocab < (int64_t{1} << 31) && dim <= (int64_t{1} << 30) &&
         (tokens + 31) / 32 * ((dim + 63) / 64) <= kMaxGrid;
}

bool embed_few(const EmbedArgs &a) { return a.tokens <= kFewTokens; }

size_t embed_work_bytes(int64_t tokens, int64_t dim) {
  if (tokens == 0) return 0;
  const int chunk = chunk_of(tokens, dim);
  const size_t b = up256(static_cast<size_t>(tokens) * 4);
  return 2 * b * (tokens > kSortTile ? 2 : 1) +
         up256(static_cast<size_t>((tokens + chunk - 1) / chunk) * 2 * static_cast<size_t>(dim) * 4);
}

void launch_embed_lookup(const EmbedArgs &a, hipStream_t s) {
  // whole vectors of eight columns where every row of the table and of the output starts on 16 bytes
  const bool vec = a.dim % 8 == 0 && a.ldo % 8 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
  const int64_t per_row = vec ? a.dim / 8 : a.dim;
  int lanes_log2 = 3;
  while (lanes_log2 < 8 && (int64_t{1} << lanes_log2) < per_row) ++lanes_log2;
  const int64_t rows = int64_t{1} << (8 - lanes_log2);
  const dim3 grid((a.tokens + rows - 1) / rows);
  if (a.value_bf16) {
    if (vec) lookup_kernel<uint16_t, 8><<<grid, kBlock, 0, s>>>(a, lanes_log2);
    else lookup_kernel<uint16_t, 1><<<grid, kBlock, 0, s>>>(a, lanes_log2);
  } else {
    if (vec) lookup_kernel<float, 8><<<grid, kBlock, 0, s>>>(a, lanes_log2);
    else lookup_kernel<float, 1><<<grid, kBlock, 0, s>>>(a, lanes_log2);
  }
}

void launch_embed_order(const EmbedArgs &a, hipStream_t s) {
  const Order o = order_of(a);
  const int sort_blocks = embed_few(a) ? 0 : static_cast<int>((a.tokens + kSortTile - 1) / kSortTile);
  const int64_t zero_bytes = a.accumulate ? 0 : a.vocab * a.dim * (a.grad_bf16 ? 2 : 4);
  const int64_t want = (zero_bytes / 16 + kSortThreads - 1) / kSortThreads;
  const int zero_blocks = zero_bytes == 0 ? 0 : static_cast<int>(want < 1 ? 1 : want > 1024 ? 1024 : want);
  const dim3 grid(static_cast<unsigned>(sort_blocks + zero_blocks));
  int bits = 1;
  while ((a.vocab >> bits) > 0) ++bits;
  if (bits <= 32 - kSortShift)
    order_kernel<uint32_t><<<grid, kSortThreads, 0, s>>>(a, o.key[0], o.pos[0], bits, sort_blocks, zero_bytes);
  else
    order_kernel<uint64_t><<<grid, kSortThreads, 0, s>>>(a, o.key[0], o.pos[0], bits, sort_blocks, zero_bytes);
  int64_t run = kSortTile;
  for (int p = 0; p < o.passes; ++p, run *= kMergeWays)
    merge_kernel<<<dim3((a.tokens + kBlock - 1) / kBlock), kBlock, 0, s>>>(
        o.key[p & 1], o.pos[p & 1], o.key[(p + 1) & 1], o.pos[(p + 1) & 1], a.tokens, run);
}

void launch_embed_sum(const EmbedArgs &a, hipStream_t s) {
  if (a.value_bf16) {
    if (a.grad_bf16) sum_by_width<uint16_t, uint16_t>(a, s);
    else sum_by_width<uint16_t, float>(a, s);
  } else {
    if (a.grad_bf16) sum_by_width<float, uint16_t>(a, s);
    else sum_by_width<float, float>(a, s);
  }
}

}  // namespace ob
