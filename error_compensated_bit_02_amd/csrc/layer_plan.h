// How a linear layer's call runs (linear.hip): whether its few tokens go through the
// vector units, else which tiles, in how many slices of the contraction, and what
// is copied beforehand.  Plain C++ so that the host tests can check which shapes
// reach which kernel.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace ob {

struct LayerShape {
  int64_t rows, out, in;     // tokens, rows of the weight, columns of the weight
  bool f32;                  // type of x (or dy), y (dx) and what is added
  bool weight_f32;           // type of the list that holds weight and bias
  bool aligned;              // x's (dy's) rows start on 16 bytes
  bool back;                 // the input gradient
};
// How a call of this shape runs: operands packed into the workspace, tiles,
// slices of the contraction.  The workspace holds A's parts, B's and the slices' sums.
struct LayerPlan {
  bool pack_a, pack_b;       // A: the weight, B: x or dy
  int a_parts, b_parts;
  int tile, m_tiles, n_tiles, splits;
  int64_t turns_each;
  size_t a_bytes, b_bytes, part_bytes;
};

// Up to so many tokens may go through the vector units; their gradient's
// contraction is cut into slices of kLayerSlice.
constexpr int kLayerFew = 8, kLayerSlice = 1024;
// A grid holds fewer than 2^32 work-items, a workgroup up to 512 of them.
constexpr int64_t kMostGroups = 0xffffffffLL / 512;

// Tiles that are built, and their times in microseconds: of a workgroup's start and
// end, of a turn on a CU of its own and with per_cu workgroups on it.  The
// plan is the tile and the number of slices with the least time by them.  Forward /
// gradient in us with each tile's best slices, the taken one marked:
//   bf16               256 x 256    128 x 128      128 x 32
//   1024^3             30 / 31      11.6 / 11.7    8.7 / 8.6 *
//   4096 x 2048^2      44 / 44      36 / 36 *      62 / 61
//   4096^3             100 / 100 *  129 / 130      226 / 232
//   16384 2048->8192   422 / 402 *  532 / 508      918 / 965
//   fp32               128 x 128    128 x 64       128 x 64, cut on the way
//   777 2048->1000     37* / 35     41 / 34 *      45 / 43
//   256 x 2048^2       33 / 32      32 / 32        28 / 30 *
//   4096^3             703 / 668 *  860 / 770      850 / 884
//   bf16 and fp32 weights
//   64 x 4096^2        62 / 49      60 / 49        26 / 27 *
//   777 2048->1000     29* / 35     32 / 32 *      42 / 33
//   2048^3             64 / 58 *    78 / 58        77 / 84
//   fp32 and bf16 weights
//   64 x 4096^2        24 / 22      22 / 21 *      23 / 21
//   777 2048->1000     28* / 33     28 / 28 *      35 / 22
//   2048^3             64 / 68 *    70 / 63        62 / 60
//   4096^3             362 / 345 *  424 / 396      460 / 449
// Cutting on the way saves the parts' copy, whose cost the weight's size settles, and
// cuts an operand again in every tile that reads it: it wins where few tiles share it.
// One table serves both mixed types, whose times differ: fp32 x with bf16 weights is up to a
// quarter from its best tile by it.  per_cu: workgroups of a CU that the estimate
// counts on; of the tiles that cut on the way two fit and one is counted, so beyond
// 256 workgroups their estimate is too long.
struct LayerTiles {
  int features, tokens, depth, per_cu;
  bool raw;                          // fp32 as it lies
  double start, alone, full;
};
constexpr LayerTiles kPlainTiles[] = {{256, 256, 64, 1, false, 9.0, 1.40, 1.40}, {128, 128, 64, 2, false, 4.5, 0.60, 1.0}, {128, 32, 64, 2, false, 4.0, 0.40, 0.55}};
constexpr LayerTiles kSixTiles[] = {{128, 128, 32, 1, false, 5.0, 1.20, 1.25}, {128, 64, 32, 1, false, 4.0, 0.70, 0.78}, {128, 64, 32, 1, true, 4.0, 1.20, 1.20}};
constexpr LayerTiles kThreeTiles[] = {{128, 128, 32, 2, false, 5.0, 0.50, 0.85}, {128, 64, 32, 2, false, 4.0, 0.40, 0.60}, {128, 64, 32, 1, true, 4.0, 0.70, 0.70}};

// Row stride of a copied operand, and where the next section of the workspace starts.
inline int64_t layer_pitch(int64_t n) { return (n + 63) / 64 * 64; }
inline size_t layer_section(size_t n) { return (n + 255) / 256 * 256; }
inline int64_t layer_features(const LayerShape &s) { return s.back ? s.in : s.out; }
inline int64_t layer_depth(const LayerShape &s) { return s.back ? s.out : s.in; }

// Whether few tokens go through the vector units.  Their time grows with the tokens, the
// matrix units' hardly does.  Forward / gradient in us, vector units against matrix units:
//   bf16  1 token    4096 x 4096  8 / 12.5 : 13 / 13    8192 x 8192  21 / 30 : 25 / 27
//         4 tokens   4096 x 4096  8 / 14 : 13 / 13      8192 x 8192  22 / 42 : 25 / 27
//         8 tokens   2048 x 2048  8 / 13.5 : 13 / 13    4096 x 4096  12.5 / 27 : 13 / 13
//                    8192 x 8192  35 / 89 : 25 / 27
//   fp32  1 token    8192 x 8192  42 / 43 : 89 / 84
//         8 tokens   4096 x 4096  18 / 29 : 29 / 28     8192 x 8192  55 / 92 : 92 / 85
// A bf16 weight that the matrix units cannot read as it lies would be copied first.
inline bool few_by_vectors(const LayerShape &s) {
  if (s.rows > kLayerFew) return false;
  const int64_t work = s.rows * s.out * s.in;
  if (s.weight_f32) return !s.back || work <= int64_t{1} << 28;
  return s.in % 8 != 0 || work <= int64_t{1} << (s.back ? 25 : 28);
}

inline bool layer_fits(int64_t rows, int64_t out, int64_t in) {
  // a tile's 256 rows (or 64 of the weight) lie within 2 GB; tiles of 128 x 128 fit the grid
  constexpr int64_t kMost = int64_t{1} << 21;
  return rows >= 0 && rows <= (int64_t{1} << 24) && out >= 1 && out <= kMost && in >= 1 && in <= kMost &&
         ((rows + 127) / 128) * ((std::max(out, in) + 127) / 128) <= kMostGroups;
}

inline LayerPlan layer_plan(const LayerShape &s) {
  LayerPlan p{};
  const int64_t features = layer_features(s), depth = layer_depth(s);
  p.splits = 1;
  if (few_by_vectors(s)) {
    p.tile = -1;
    if (s.back) p.splits = static_cast<int>((depth + kLayerSlice - 1) / kLayerSlice);
  } else {
    p.a_parts = s.weight_f32 ? 3 : 1;
    p.b_parts = s.f32 ? 3 : 1;
    const bool raw_rows_a = !s.weight_f32 && s.in % 8 != 0, raw_rows_b = !s.f32 && (depth % 8 != 0 || !s.aligned);
    const size_t a_bytes = layer_section(static_cast<size_t>(p.a_parts) * s.out * layer_pitch(s.in) * 2);
    const size_t b_bytes = layer_section(static_cast<size_t>(p.b_parts) * s.rows * layer_pitch(depth) * 2);
    const int products = p.a_parts * p.b_parts;
    const LayerTiles *tiles = products == 1 ? kPlainTiles : products == 9 ? kSixTiles : kThreeTiles;
    const double part = static_cast<double>(s.rows) * features * 4 / 3e6;
    double best = 0.0;
    p.tile = -1;
    for (int k = 0; k < 3; ++k) {
      const int64_t m = (features + tiles[k].features - 1) / tiles[k].features, n = (s.rows + tiles[k].tokens - 1) / tiles[k].tokens;
      const int64_t turns = (depth + tiles[k].depth - 1) / tiles[k].depth, most = m * n >= 512 ? 1 : std::min<int64_t>(turns, 64);      // no slices where the tiles fill the card
      // packing: its launch, and ten bytes read and written an fp32 element (four a bf16 one)
      const bool pack_a = raw_rows_a || (s.weight_f32 && !tiles[k].raw), pack_b = raw_rows_b || (s.f32 && !tiles[k].raw);
      const double packing = (pack_a || pack_b ? 4.0 : 0.0) + (pack_a ? a_bytes / 3.5e6 : 0.0) + (pack_b ? b_bytes / 3.5e6 : 0.0);
      for (int64_t want = 1; want <= most; ++want) {
        const int64_t each = (turns + want - 1) / want, splits = (turns + each - 1) / each, groups = m * n * splits;
        if (splits != want || groups > kMostGroups) continue;
        double t = packing + tiles[k].start + (splits > 1 ? 4.0 + splits * part : 0.0);
        const int64_t held = 256 * tiles[k].per_cu;
        if (groups <= 256) t += each * tiles[k].alone;
        else t += static_cast<double>((groups + held - 1) / held) * each * tiles[k].full;
        if (p.tile < 0 || t < best) {
          best = t;
          p.tile = k;
          p.m_tiles = static_cast<int>(m);
          p.n_tiles = static_cast<int>(n);
          p.splits = static_cast<int>(splits);
          p.turns_each = each;
          p.pack_a = pack_a;
          p.pack_b = pack_b;
        }
      }
    }
    p.a_bytes = p.pack_a ? a_bytes : 0;
    p.b_bytes = p.pack_b ? b_bytes : 0;
  }
  p.part_bytes = p.splits > 1 ? layer_section(static_cast<size_t>(p.splits) * s.rows * ((features + 3) / 4 * 4) * 4) : 0;
  return p;
}

}  // namespace ob
