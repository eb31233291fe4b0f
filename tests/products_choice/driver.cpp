// Prints what products_choice.h picks.  Lines on standard input:
//   fp8 m n k tile          -> tiling (-1: the kernel for few rows)
//   gated rows d f          -> tilings of the forward pass (-1), of dx, of dw; parts of dx
//   grids                   -> the most threads that any launch asks for, over sizes at and near the limits
#include <cstdio>
#include <cstring>

#include "products_choice.h"

namespace {

using namespace opt8;

constexpr int64_t kMaxCount = int64_t{1} << 22, kMaxWidth = int64_t{1} << 20, kMaxElements = int64_t{1} << 37;

int fp8_threads(int choice) {
  const int threads[kTileChoices] = {512, 256, 512, 256, 512};
  return threads[choice];
}
int gated_threads(int choice) {
  const int threads[kTileChoices] = {256, 256, 512, 256, 512};
  return threads[choice];
}

// 1, 2, and a power of two, the number below and the one above, up to `most`
template <class F>
void sizes(int64_t most, F&& f) {
  for (int64_t p = 1; p <= most; p *= 2)
    for (int64_t v = p - 1; v <= p + 1; ++v)
      if (v >= 1 && v <= most) f(v);
}

int64_t worst = 0;
void launched(int64_t blocks, int64_t threads) { worst = std::max(worst, blocks * threads); }

void grids() {
  sizes(kMaxCount, [&](int64_t m) {
    sizes(kMaxCount, [&](int64_t n0) {
      // as many columns as the count of elements leaves, too
      for (int64_t n : {n0, std::min(kMaxCount, kMaxElements / m)}) {
        if (m * n > kMaxElements) continue;
        launched(tiles_of(m, n, 128), 256);      // quantiser
        for (int64_t k : {int64_t{0}, int64_t{1}, int64_t{129}, int64_t{4096}, kMaxElements / std::max(m, n)}) {
          if (m <= kFewRows) launched((n + 15) / 16, 256);
          for (bool tile : {false, true}) {
            const int c = fp8_choice(m, n, std::min(k, kMaxCount), tile);
            launched(tiles_of(m, n, tile_size(c)), fp8_threads(c));
          }
          const int64_t d = std::min(std::max<int64_t>(k, 1), kMaxWidth);
          if (n > kMaxWidth || m * d > kMaxElements || n * d > kMaxElements) continue;
          const int64_t rows = m, f = n;
          int c = gated_forward_choice(rows, d, f);
          launched(((rows + tile_size(c) - 1) / tile_size(c)) * ((f + tile_size(c) / 2 - 1) / (tile_size(c) / 2)), gated_threads(c));
          launched((f + 15) / 16, 256);
          c = gated_dx_choice(rows, d, f);
          launched(tiles_of(rows, d, tile_size(c)) * gated_dx_splits(rows, d, f), gated_threads(c));
          if (gated_dx_splits(rows, d, f) > 1) launched((rows * d + 255) / 256, 256);
          c = gated_dw_choice(rows, d, f);
          launched(2 * tiles_of(f, d, tile_size(c)), gated_threads(c));
          // the same with the widths as the large dimension of x and of the weights
          c = gated_dx_choice(rows, f, d);
          launched(tiles_of(rows, f, tile_size(c)) * gated_dx_splits(rows, f, d), gated_threads(c));
        }
      }
    });
  });
}

}  // namespace

int main() {
  char what[16];
  while (std::scanf("%15s", what) == 1) {
    long long a, b, c, d;
    if (!std::strcmp(what, "fp8")) {
      if (std::scanf("%lld %lld %lld %lld", &a, &b, &c, &d) != 4) return 1;
      std::printf("%d\n", a <= kFewRows ? -1 : fp8_choice(a, b, c, d != 0));
    } else if (!std::strcmp(what, "gated")) {
      if (std::scanf("%lld %lld %lld", &a, &b, &c) != 3) return 1;
      std::printf("%d %d %d %d\n", a <= kFewRows ? -1 : gated_forward_choice(a, b, c), gated_dx_choice(a, b, c),
                  gated_dw_choice(a, b, c), gated_dx_splits(a, b, c));
    } else if (!std::strcmp(what, "grids")) {
      grids();
      std::printf("%lld\n", static_cast<long long>(worst));
    } else {
      return 1;
    }
  }
  return 0;
}
