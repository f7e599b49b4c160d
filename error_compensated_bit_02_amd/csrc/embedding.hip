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
//  1. order: each workgroup sorts one tile of kSortTile tokens in LDS (a
//     bitonic network on id and position packed in one key, so the order is
//     total), while the other workgroups of the same launch zero the
//     gradient, which has to be written whole and usually takes longer;
//  2. merge: runs of sorted tiles are merged kMergeWays at a time; an
//     element's place is its index in its own run plus its rank in each
//     other run, found by binary search;
//  3. sum: one wavefront sums kRun consecutive sorted tokens of one slice
//     of columns in fp32; a run of equal ids inside the chunk is written out,
//     the parts of a run that crosses chunks go to the workspace;
//  4. join: the chunk where such a run begins adds its parts in order.
#include "internal.h"

#pragma clang fp contract(off)

namespace ob {
namespace {

constexpr int kSortTile = 4096;
constexpr int kSortThreads = 1024;
constexpr int kSortShift = 12;          // log2(kSortTile)
constexpr int kMergeWays = 16;
constexpr int kRun = 32;                // sorted tokens summed by one wavefront
constexpr uint32_t kNoId = 0xffffffffu; // sorts last, never summed

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  bf16x2 r;
  r[0] = static_cast<__bf16>(a);
  r[1] = static_cast<__bf16>(b);
  return __builtin_bit_cast(uint32_t, r);
}

// N consecutive elements as fp32 and back: one vector access each where N > 1
// (the caller has checked alignment).
template <typename T, int N>
struct Vec {
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
  int64_t chunks;
  int passes;            // merge passes; the result is in key/pos[passes & 1]
};

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
  o.chunks = (a.tokens + kRun - 1) / kRun;
  return o;
}

// K: uint32_t while an id and a place in the tile fit in 32 bits, else uint64_t.
template <typename K>
__global__ __launch_bounds__(kSortThreads) void order_kernel(const EmbedArgs a, uint32_t *key, uint32_t *pos,
                                                             int sort_blocks, int64_t zero_bytes) {
  if (static_cast<int>(blockIdx.x) >= sort_blocks) {   // zero the gradient
    const int64_t n = zero_bytes / 16;
    uint4 *g = static_cast<uint4 *>(a.grad);
    const int64_t step = static_cast<int64_t>(gridDim.x - sort_blocks) * kSortThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x - sort_blocks) * kSortThreads + threadIdx.x;
    for (int64_t i = first; i < n; i += step) g[i] = make_uint4(0, 0, 0, 0);
    // the last bytes of a gradient that ends inside 16 bytes, two at a time (padding stays untouched)
    if (first < (zero_bytes - n * 16) / 2) reinterpret_cast<uint16_t *>(g + n)[first] = 0;
    return;
  }
  __shared__ K s[kSortTile];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortTile;
  const int len = static_cast<int>(min(static_cast<int64_t>(kSortTile), a.tokens - base));
  int n2 = 64;
  while (n2 < len) n2 *= 2;
  const K none = static_cast<K>(a.vocab);   // the id behind the table's last
  for (int i = threadIdx.x; i < n2; i += kSortThreads) {
    K k = ~K{0};
    if (i < len) {
      const int64_t id = id_at(a, base + i);
      k = ((id >= 0 && id < a.vocab ? static_cast<K>(id) : none) << kSortShift) | static_cast<K>(i);
    }
    s[i] = k;
  }
  __syncthreads();
  for (int size = 2; size <= n2; size *= 2) {
    for (int stride = size / 2; stride > 0; stride /= 2) {
      for (int p = threadIdx.x; p < n2 / 2; p += kSortThreads) {
        const int i = 2 * stride * (p / stride) + (p & (stride - 1));
        const K x = s[i], y = s[i + stride];
        if ((x > y) == ((i & size) == 0)) {
          s[i] = y;
          s[i + stride] = x;
        }
      }
      __syncthreads();
    }
  }
  for (int i = threadIdx.x; i < len; i += kSortThreads) {
    const K k = s[i];
    const K id = k >> kSortShift;
    key[base + i] = id == none ? kNoId : static_cast<uint32_t>(id);
    pos[base + i] = static_cast<uint32_t>(base) + static_cast<uint32_t>(k & (kSortTile - 1));
  }
}

// Merges kMergeWays sorted runs of `run` elements each.
__global__ __launch_bounds__(kBlock) void merge_kernel(const uint32_t *key, const uint32_t *pos, uint32_t *key_out,
                                                       uint32_t *pos_out, int64_t tokens, int64_t run) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  if (j >= tokens) return;
  const uint32_t k = key[j];
  const int64_t mine = j / run, first = mine / kMergeWays * kMergeWays;
  int64_t place = j - (mine - first) * run;
  uint32_t top = 1;                        // smallest power of two past the run's length
  while (top <= run) top *= 2;
#pragma unroll 1
  for (int h = 0; h < kMergeWays; h += 8) {
    int64_t start[8];
    uint32_t len[8], below[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t b = first + h + u;
      start[u] = b * run;
      const int64_t left = tokens - start[u];
      len[u] = b == mine || left <= 0 ? 0u : static_cast<uint32_t>(min(left, run));
      below[u] = 0;                        // elements known to come before (k, this run)
    }
    for (uint32_t step = top / 2; step > 0; step /= 2) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t probe = below[u] + step;
        if (probe <= len[u]) {
          const uint32_t other = key[start[u] + probe - 1];
          if (first + h + u < mine ? other <= k : other < k) below[u] = probe;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) place += below[u];
  }
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
                                                     float *part, int64_t chunks, int slices) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= chunks * slices) return;
  const int64_t chunk = unit / slices;
  const int64_t c = (static_cast<int64_t>(unit - chunk * slices) * 64 + lane) * N;
  const bool live = c < a.dim;
  const int64_t j0 = chunk * kRun;
  const int len = static_cast<int>(min(static_cast<int64_t>(kRun), a.tokens - j0));
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
      const uint32_t p = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(lp), (b + u) & (kRun - 1)));
      Vec<T, N>::load(dy + static_cast<int64_t>(p) * a.lddy, v[u]);   // absent tokens read token 0, unused
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
                                                      int64_t chunks, int slices) {
  const int64_t chunk = blockIdx.x / slices;
  const int64_t j0 = chunk * kRun, j1 = j0 + kRun;
  if (j1 >= a.tokens) return;
  const uint32_t k = key[j1 - 1];
  if (k == kNoId || key[j1] != k) return;
  if (key[j0] == k && j0 > 0 && key[j0 - 1] == k) return;    // began earlier
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (static_cast<int64_t>(blockIdx.x - chunk * slices) * 64 + lane) * N;
  const bool live = c < a.dim;
  int64_t lo = j1, hi = a.tokens;                            // first position past the run
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (key[mid] == k) lo = mid + 1;
    else hi = mid;
  }
  const int64_t parts = (lo - 1) / kRun - chunk;             // later chunks that hold a part
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

template <typename T, typename G, int N>
void sum_one(const EmbedArgs &a, hipStream_t s) {
  const Order o = order_of(a);
  const int slices = static_cast<int>((a.dim + 64 * N - 1) / (64 * N));
  const int side = o.passes & 1;
  const int64_t units = o.chunks * slices;
  sum_kernel<T, G, N><<<dim3((units + kWaves - 1) / kWaves), kBlock, 0, s>>>(a, o.key[side], o.pos[side], o.part,
                                                                             o.chunks, slices);
  if (o.chunks > 1) join_kernel<G, N><<<dim3(units), kBlock, 0, s>>>(a, o.key[side], o.part, o.chunks, slices);
}

template <typename T, typename G>
void sum_by_width(const EmbedArgs &a, hipStream_t s) {
  // eight columns a lane where every row of dy and of the gradient starts on 16 bytes
  if (a.dim % 8 == 0 && a.lddy % 8 == 0 && reinterpret_cast<uintptr_t>(a.dy) % 16 == 0) sum_one<T, G, 8>(a, s);
  else sum_one<T, G, 1>(a, s);
}

}  // namespace

bool embed_fits(int64_t tokens, int64_t vocab, int64_t dim) {
  // ids are 32-bit; the lookup has a workgroup a token at most, the join one per chunk and slice
  const int64_t slices = (dim + 63) / 64;
  return tokens <= kMaxGrid && vocab < (int64_t{1} << 31) && dim < (int64_t{1} << 31) &&
         (tokens + kRun - 1) / kRun <= kMaxGrid / slices;
}

size_t embed_work_bytes(int64_t tokens, int64_t dim) {
  if (tokens == 0) return 0;
  const size_t b = up256(static_cast<size_t>(tokens) * 4);
  return 2 * b * (tokens > kSortTile ? 2 : 1) +
         up256(static_cast<size_t>((tokens + kRun - 1) / kRun) * 2 * static_cast<size_t>(dim) * 4);
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
  const int sort_blocks = static_cast<int>((a.tokens + kSortTile - 1) / kSortTile);
  const int64_t zero_bytes = a.accumulate ? 0 : a.vocab * a.dim * (a.grad_bf16 ? 2 : 4);
  const int64_t want = (zero_bytes / 16 + kSortThreads - 1) / kSortThreads;
  const int zero_blocks = zero_bytes == 0 ? 0 : static_cast<int>(want < 1 ? 1 : want > 1024 ? 1024 : want);
  if (sort_blocks + zero_blocks == 0) return;
  const dim3 grid(static_cast<unsigned>(sort_blocks + zero_blocks));
  if ((a.vocab + 1) < (int64_t{1} << (32 - kSortShift)))
    order_kernel<uint32_t><<<grid, kSortThreads, 0, s>>>(a, o.key[0], o.pos[0], sort_blocks, zero_bytes);
  else
    order_kernel<uint64_t><<<grid, kSortThreads, 0, s>>>(a, o.key[0], o.pos[0], sort_blocks, zero_bytes);
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
