// Checks of matrices and sizes that the operators' C entry points share
// (products_host.cpp, layers_host.cpp).
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include <hip/hip_runtime.h>

#include "../../include/opt8_products.h"
#include "opt8_error.h"

namespace opt8 {

__attribute__((format(printf, 2, 3))) inline int refuse(int code, const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  return set_last_error(code, text);
}

// The kernels index rows and columns in 32 bits and a tile's rows by 32-bit byte
// offsets (256 * 2^23 = 2^31).  A launch has fewer than 2^32 threads: at 2^37 results
// the quantiser's has 2^31 (128 x 128 to 256 threads), the products' 2^30 (256 x
// 256 to 512 or 256 threads: smaller tiles, which would take up to 2^35, are never
// chosen there), all others stay below 2^29.
constexpr int64_t kMaxCount = int64_t{1} << 22;
constexpr int64_t kMaxWidth = int64_t{1} << 20;
constexpr int64_t kMaxElements = int64_t{1} << 37;
constexpr int64_t kMaxRowBytes = int64_t{1} << 23;
constexpr int64_t kMaxDistance = int64_t{1} << 38;    // of rows; kMaxCount of them span 2^62 bytes

inline int type_bytes(int type) {
  switch (type) {
    case OPT8_TYPE_BF16:
    case OPT8_TYPE_FP16: return 2;
    case OPT8_TYPE_FP32: return 4;
    default: return 1;
  }
}

struct Matrix {
  const char* name;
  const void* p;
  int64_t rows, cols, ld;
  int size;
  bool output;
  bool core;     // feeds the matrix cores: 16-byte rows
};

// Bytes from the first to past the last element.
inline int64_t span(const Matrix& x) { return ((x.rows - 1) * x.ld + x.cols) * x.size; }

// Whether two matrices share a byte.  Spans that meet are still apart where both
// have the same distance between rows and their columns lie side by side in it
// (two halves of one wider matrix).
inline bool overlap(const Matrix& x, const Matrix& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  if (a + span(x) <= b || b + span(y) <= a) return false;
  const int64_t pitch = x.ld * x.size;
  if (pitch != y.ld * y.size) return true;
  const int64_t wx = x.cols * x.size, wy = y.cols * y.size;
  int64_t at = static_cast<int64_t>(b - a) % pitch;     // where y's row starts in x's
  if (at < 0) at += pitch;
  return at < wx || at + wy > pitch;
}

inline int check_count(const char* name, int64_t v, int64_t low, int64_t high) {
  if (v < low || v > high)
    return refuse(OPT8_E_SIZE, "%s must be %lld to %lld (got %lld)", name, static_cast<long long>(low),
                  static_cast<long long>(high), static_cast<long long>(v));
  return OPT8_OK;
}

// Matrices with no pointer are absent; the rest are checked one by one, then
// outputs against all others.
inline int check_matrices(const Matrix* list, int n) {
  for (int i = 0; i < n; ++i) {
    const Matrix& x = list[i];
    if (!x.p) continue;
    if (x.ld < x.cols)
      return refuse(OPT8_E_SIZE, "%s: ld %lld is below its %lld columns", x.name, static_cast<long long>(x.ld),
                    static_cast<long long>(x.cols));
    if (x.ld > kMaxDistance || (x.core && x.ld * x.size > kMaxRowBytes))
      return refuse(OPT8_E_SIZE, "%s: ld %lld is too large", x.name, static_cast<long long>(x.ld));
    if (x.rows * x.cols > kMaxElements)
      return refuse(OPT8_E_SIZE, "%s: over 2^37 elements", x.name);
    const uintptr_t at = reinterpret_cast<uintptr_t>(x.p);
    if (x.core && (at % 16 || x.ld * x.size % 16))
      return refuse(OPT8_E_ALIGN, "%s: must start on 16 bytes and have rows a multiple of 16 bytes apart", x.name);
    if (at % static_cast<uintptr_t>(x.size)) return refuse(OPT8_E_ALIGN, "%s: not aligned to its elements", x.name);
  }
  for (int i = 0; i < n; ++i) {
    if (!list[i].p || !list[i].output || list[i].rows <= 0 || list[i].cols <= 0) continue;
    for (int j = 0; j < n; ++j) {
      if (j == i || !list[j].p || list[j].rows <= 0 || list[j].cols <= 0) continue;
      if (overlap(list[i], list[j])) return refuse(OPT8_E_ALIAS, "%s overlaps %s", list[i].name, list[j].name);
    }
  }
  return OPT8_OK;
}

inline int launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return refuse(OPT8_E_HIP, "%s: kernel launch failed: %s", what, hipGetErrorString(e));
  return OPT8_OK;
}

inline int64_t blocks(int64_t n) { return (n + OPT8_FP8_BLOCK - 1) / OPT8_FP8_BLOCK; }

}  // namespace opt8
