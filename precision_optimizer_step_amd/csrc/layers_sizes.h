// How the operators in opt8_layers.h cut their work and their workspaces: pure
// functions of the sizes, without HIP, so that a host program can ask them too.
#pragma once

#include <algorithm>
#include <cstdint>

namespace opt8 {

inline int64_t pieces_of(int64_t n, int64_t each) { return (n + each - 1) / each; }
inline int64_t align16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// Whether a call that moves so many bytes reads its 16-bit rows past the caches: where
// the last-level cache (256 MB) cannot hold them for the next reader.  16384 x 4096
// with both kinds of loads: norm with residual and codes 109 us through the caches, 100
// past them; its backward pass 101 and 94; embedding's gradient 107 and 97; norm of
// 2.65G gradients 878 and 781.  Small calls repeated on inputs that stayed in the cache:
// 64032 x 128 norms 6.9 and 7.6 us, 4001 x 1600 backward 15.0 and 17.4.
inline bool streams(int64_t bytes) { return bytes > int64_t{128} << 20; }

// Whether the norm's 16-bit y is stored through the caches, for a product that reads it
// again for each of its tiles.  Norm and gated block in a row, y through the caches and
// past them, us:  4096 wide, f 4096:  64 rows: 24.0 28.5   333: 39.1 52.0   1000: 64.6 70.4
//   1500: 89.5 93.2   1750: 97.0 98.2   2048: 105.8 105.4   4096: 211 213;  1024 wide:
//   333: 16.7 19.3   1500: 32.1 33.8   4000: 68.5 69.5   6000: 100.3 99.9.  The norm alone:
//   333 x 4096: 4.2 3.8   2048: 12.8 11.3   16384: 98.8 91.6.  (A reader that takes
// a result once does not mind: lookup and norm 6.8 and 6.9 at 333 rows, 10.6 and 9.6 at 1000.)
inline bool stays(int64_t bytes) { return bytes <= int64_t{8} << 20; }

// ---------------------------------------------------------------- embedding's gradient
// Tokens whose like a wave finds by itself (two in each lane), with no sort.  Whole calls
// in us, so and with the sort (bf16):  1 x 4096 added: 6.1 8.3   15 x 97 added: 6.0 13.5
//   128 x 4096 added: 6.5 13.9   102 x 932 into 26413 rows: 12.6 19.4   128 x 4096 into
//   50257 rows: 57.5 63.8;   of one id only, added: 64 x 4096: 10.1 12.5   128 x 4096: 19.3 13.2
constexpr int kFewTokens = 128;

// The sort's workgroups, a power of two: each owns one of every `groups` ids in a row
// (so that ids next to each other, which are often the frequent ones, are not one
// workgroup's), at most kSortRange of them, counted in LDS.
constexpr int kSortWaves = 16;
constexpr int kSortRange = 1024;
struct SortShape {
  int groups, shift, range;    // groups = 1 << shift
};
inline SortShape sort_shape(int64_t vocab) {
  SortShape s{256, 8, 0};
  while (pieces_of(vocab, s.groups) > kSortRange) s.groups *= 2, ++s.shift;
  s.range = static_cast<int>(pieces_of(vocab, s.groups));
  return s;
}

// Sorted tokens that a wave adds up: 32 where that leaves at least 4096 waves (4 to a
// SIMD), fewer for short batches; at most 32 (a wave keeps a chunk's tokens and its two
// neighbours in its lanes).  Measured, whole calls in us with chunks of 8, 16 and 32
// (50257 ids, bf16):  1001 x 1600: 16.1 19.7 27.4   4096 x 1024: 20.8 25.3 33.5
//   4096 x 4096: 27.7 29.2 35.6   16384 x 1024: 36.0 35.4 40.6   8192 x 4096: 48.0 44.5 49.1
//   65536 x 1024: 99.3 85.2 80.1   16384 x 4096: 101.8 97.3 95.3
inline int64_t sum_chunk(int64_t tokens, int64_t d) {
  const int64_t waves = tokens * pieces_of(d, 512);
  return waves >= 32 * 4096 ? 32 : waves >= 16 * 4096 ? 16 : 8;
}

struct EmbeddingSpace {
  int64_t order, keys, starts, partial, bytes;    // offsets
};
inline EmbeddingSpace embedding_space(int64_t tokens, int64_t vocab, int64_t d) {
  EmbeddingSpace s;
  s.order = 0;
  s.keys = align16(4 * tokens);
  s.starts = s.keys + align16(4 * tokens);
  const SortShape sort = sort_shape(vocab);
  s.partial = s.starts + align16(4 * (int64_t{sort.groups} * sort.range + 1));
  // two sums of each chunk: of the id that it shares with the one before, and with the one behind
  s.bytes = s.partial + align16(8 * d * pieces_of(tokens, sum_chunk(tokens, d)));
  return s;
}

// ---------------------------------------------------------------- norm's backward pass
// Lanes that share a row, and pieces of 8 values that each of them holds.
struct RowShape {
  int lanes, pieces;
};
constexpr int64_t kNormHeld = 16384;    // longer rows are read twice
inline RowShape norm_grad_shape(int64_t d) {
  if (d <= 128) return {16, 1};
  if (d <= 512) return {64, 1};
  if (d <= 1024) return {64, 2};
  if (d <= 2048) return {256, 1};
  if (d <= 4096) return {256, 2};
  if (d <= 8192) return {1024, 1};
  return {1024, 2};
}
// Workgroups that each keep a sum of dweight, and so rows of the workspace: two to a CU.
// Both kernels in us with 256, 384, 512, 768 and 1024 of them:  16384 x 4096 bf16 with dsum:
// 126 98.7 95.7 99.1 110   16384 x 2048: 89 65 55.4 52.3 54.9   4001 x 1600 fp16: 21.4 17.1
//   15.5 14.8 15.5   64032 x 128: 20.0 16.6 15.3 15.1 15.7   500 x 4096: 10.5 11.1 12.1 12.1 12.1
inline int64_t norm_grad_groups(int64_t rows, int64_t d) {
  if (d > kNormHeld) return std::max<int64_t>(1, std::min<int64_t>(64, rows / 8));
  const int64_t lanes = norm_grad_shape(d).lanes;
  const int64_t at_once = lanes <= 256 ? 256 / lanes : 1;      // rows to a workgroup at a time
  const int64_t most = lanes <= 256 ? 512 : 256;
  return std::max<int64_t>(1, std::min<int64_t>(most, pieces_of(rows, at_once)));
}
inline int64_t norm_grad_space(int64_t rows, int64_t d) {
  return rows <= 0 ? 0 : align16(4 * d * norm_grad_groups(rows, d));
}

// ---------------------------------------------------------------- gradients' norm
// Workgroups, 4 to a CU.  With 512, 768, 1024, 1536 and 2048 of them, in us:  355M fp32
// values, norm and clipping to bf16: 701 625 608 624 635;  2.65G bf16 values, norm only: 1038 801
// 784 776 804.
constexpr int64_t kGradGroups = 1024;

}  // namespace opt8
