// Internal interface between the host side (products_host.cpp) and the kernels
// of the operators in opt8_products.h (fp8_quantize.hip, fp8_product.hip,
// gated_ffn.hip).  Not part of the public ABI.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

#include "../../include/opt8_products.h"

namespace opt8 {

// Queues a kernel that takes one structure.  The status is this launch's own: the
// runtime's last error may be one that an earlier call of the caller's left, which
// is the caller's to read.
template <class P>
inline hipError_t queue(void (*kernel)(P), dim3 grid, unsigned threads, hipStream_t stream, P& p) {
  void* arguments[] = {&p};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), arguments, 0, stream);
  if (e != hipSuccess) (void)hipGetLastError();    // reported by the call: not a second time by the next reader
  return e;
}

// Each queues its launches for validated, non-empty arguments.
hipError_t launch_fp8_quantize(const opt8_fp8_quant& q, hipStream_t stream);
hipError_t launch_fp8_matmul(const opt8_fp8_product& p, hipStream_t stream);
hipError_t launch_gated_ffn_forward(const opt8_gated_ffn& f, hipStream_t stream);
hipError_t launch_gated_ffn_backward(const opt8_gated_ffn_grad& g, hipStream_t stream);

// The backward pass's workspace: dg and du side by side in rows of twice
// gated_width(f) (f rounded up to whole steps of the contraction, the rest
// zeros), 16 bits each; then dx in fp32 once for each part that its long
// contraction (2f) is cut into where dx is too small to give every CU a tile.
inline int64_t gated_width(int64_t f) { return (f + 63) / 64 * 64; }
inline int64_t gated_bytes(int64_t rows, int64_t f) { return rows * 2 * gated_width(f) * 2; }
// Parts of dx: as many as fill 256 CUs with 64 x 64 tiles, at least 16 steps each.
// rows 500, d 1024, f 4096: 2 parts; 64, 4096, 16384: 4 parts.
inline int gated_dx_splits(int64_t rows, int64_t d, int64_t f) {
  const int64_t tiles = ((rows + 63) / 64) * ((d + 63) / 64), steps = 2 * gated_width(f) / 64;
  if (tiles == 0) return 1;
  int64_t parts = 256 / tiles;
  if (parts > steps / 16) parts = steps / 16;
  return static_cast<int>(parts < 1 ? 1 : parts > 16 ? 16 : parts);
}
inline int64_t gated_workspace(int64_t rows, int64_t d, int64_t f) {
  const int splits = gated_dx_splits(rows, d, f);
  return gated_bytes(rows, f) + (splits > 1 ? splits * ((rows * d + 3) / 4 * 4) * 4 : 0);
}

// Microseconds that `tiles` tiles of `steps` steps take, `at_once` of them side by
// side on the chip: a full round runs steps * step + fixed, a last round of at
// most 256 tiles (one to a CU) steps * step_few + fixed_few.
inline double estimate(int64_t tiles, int64_t steps, int at_once, double step, double fixed, double step_few, double fixed_few) {
  const int64_t rest = tiles % at_once;
  const double full = static_cast<double>(steps) * step + fixed;
  const double last = rest == 0 ? 0.0 : rest <= 256 ? static_cast<double>(steps) * step_few + fixed_few : full;
  return static_cast<double>(tiles / at_once) * full + last;
}

}  // namespace opt8
