// Which kernel a product runs in, and how the gated block's workspace is cut: pure
// functions of the sizes, without HIP, so that a host program can ask them too.
#pragma once

#include <algorithm>
#include <cstdint>

namespace opt8 {

// The tilings that the tiled products are built in: results to a workgroup, and
// teams of waves that split k inside it.
enum TileChoice : int { kTile256 = 0, kTile128, kTile128Teams2, kTile64Teams2, kTile64Teams4, kTileChoices };

inline int tile_size(int choice) { return choice == kTile256 ? 256 : choice <= kTile128Teams2 ? 128 : 64; }
inline int64_t tiles_of(int64_t m, int64_t n, int64_t size) { return ((m + size - 1) / size) * ((n + size - 1) / size); }

// Microseconds that `tiles` tiles of `steps` steps take, `at_once` of them side by
// side on the chip: a full round runs steps * step + fixed, a last round of at
// most 256 tiles (one to a CU) steps * step_few + fixed_few.
inline double estimate(int64_t tiles, int64_t steps, int at_once, double step, double fixed, double step_few, double fixed_few) {
  const int64_t rest = tiles % at_once;
  const double full = static_cast<double>(steps) * step + fixed;
  const double last = rest == 0 ? 0.0 : rest <= 256 ? static_cast<double>(steps) * step_few + fixed_few : full;
  return static_cast<double>(tiles / at_once) * full + last;
}

// The 8-bit product of more than kFewRows rows: the tiling that the estimate calls
// fastest.  Its constants fit these measurements (us at n = 4096, k = 4096 unless
// named; scales of b by TILE, and by ROW where it differs; the kernels from left to
// right):
//                     256x256    128x128   128x128, 2 teams   64x64, 2 teams   64x64, 4 teams
//   m =  128             43         21           19                10.8             10.4
//   m =  512             44         25           21                17.1             23
//   m = 1024             46         27           25                32               47
//   m = 2048             50/66      38/43        48                62               90
//   m = 4096             62/75      74/83        96               119              174
//   8192 x 8192         244/299    286/327      356               466              670
//   8192 x 8192, k 512   56         65          107               128              300
inline int fp8_choice(int64_t m, int64_t n, int64_t k, bool tile) {
  const int64_t steps = (k + 127) / 128;
  const double cost[kTileChoices] = {
      estimate(tiles_of(m, n, 256), steps, 256, tile ? 1.9 : 2.3, 4, tile ? 1.45 : 1.95, 4),
      estimate(tiles_of(m, n, 128), steps, 512, tile ? 1.12 : 1.26, 3, 0.78, 3),
      estimate(tiles_of(m, n, 128), steps, 256, 0.70, 3, 0.68, 3),
      estimate(tiles_of(m, n, 64), steps, 512, 0.50, 1.5, 0.32, 1.5),
      estimate(tiles_of(m, n, 64), steps, 256, 0.29, 1.5, 0.28, 1.5),
  };
  return static_cast<int>(std::min_element(cost, cost + kTileChoices) - cost);
}

// The gated block's products, `products` of them of m x n results and k long.  The
// constants fit these measurements (us; dx is m x n = rows x d, k = 2f):
//                                     256     128   128x2 teams  64x2   64x4
//   dx   500 x 1024, k  8192          151      84        65       48     38
//   dx  2048 x 1024, k  8192          152      86        68       57     78
//   dx  2048 x 2560, k 20480          366     251       350      395    531
//   dx  4096 x 4096, k  8192          195     242       288      414    577
//   dw  8192 x 1024, k   500           21      15        19       28     45
//   h    500 x 8192, k  1024           28      14        14       19     30
//   h   8192 x 32768, k 4096         1641    2134      3074     3956   6194
inline int gated_choice(int64_t m, int64_t n, int64_t k, int64_t products) {
  const int64_t steps = (k + 63) / 64;
  const double cost[kTileChoices] = {
      estimate(products * tiles_of(m, n, 256), steps, 256, 1.5, 11, 1.3, 11),
      estimate(products * tiles_of(m, n, 128), steps, 512, 0.97, 7, 0.66, 5),
      estimate(products * tiles_of(m, n, 128), steps, 256, 0.52, 6, 0.50, 6),
      estimate(products * tiles_of(m, n, 64), steps, 512, 0.40, 3.5, 0.34, 3),
      estimate(products * tiles_of(m, n, 64), steps, 256, 0.285, 3.5, 0.28, 3.5),
  };
  return static_cast<int>(std::min_element(cost, cost + kTileChoices) - cost);
}

// At most this many rows (single tokens) take the kernels without LDS.  8-bit: k =
// 16384, one row: 12.5 us against 30.5 of the 64x64 tiles; 16 rows: 17.3 against
// 31.0.  At 16 rows, n = 16384 and k = 4096 the tiles are the faster ones (14.9 against
// 16.7 us): a corner that the rule gives up.
constexpr int64_t kFewRows = 16;

// The backward pass's workspace: dg and du side by side in rows of twice
// gated_width(f) (f rounded up to whole steps of the contraction, the rest
// zeros), 16 bits each; then dx in fp32 once for each part that its long
// contraction (2f) is cut into where dx is too small to give every CU a tile.
inline int64_t gated_width(int64_t f) { return (f + 63) / 64 * 64; }
inline int64_t gated_bytes(int64_t rows, int64_t f) { return rows * 2 * gated_width(f) * 2; }
// Parts of dx: as many as fill 256 CUs with 64 x 64 tiles, at least 16 steps each.
// rows 500, d 1024, f 4096: 2 parts; 64, 4096, 16384: 4 parts.
inline int gated_dx_splits(int64_t rows, int64_t d, int64_t f) {
  const int64_t tiles = tiles_of(rows, d, 64), steps = 2 * gated_width(f) / 64;
  if (tiles == 0) return 1;
  const int64_t parts = std::min(256 / tiles, steps / 16);
  return static_cast<int>(parts < 1 ? 1 : parts > 16 ? 16 : parts);
}
inline int64_t gated_workspace(int64_t rows, int64_t d, int64_t f) {
  const int splits = gated_dx_splits(rows, d, f);
  return gated_bytes(rows, f) + (splits > 1 ? splits * ((rows * d + 3) / 4 * 4) * 4 : 0);
}

// The choices for the gated block's products.  The forward pass holds as many columns
// of g as of u in a tile, so its results are rows x 2f.
inline int gated_forward_choice(int64_t rows, int64_t d, int64_t f) { return gated_choice(rows, 2 * f, d, 1); }
inline int gated_dx_choice(int64_t rows, int64_t d, int64_t f) {
  const int splits = gated_dx_splits(rows, d, f);
  return gated_choice(rows, d, 2 * gated_width(f) / splits, splits);
}
inline int gated_dw_choice(int64_t rows, int64_t d, int64_t f) { return gated_choice(f, d, rows, 2); }

}  // namespace opt8
