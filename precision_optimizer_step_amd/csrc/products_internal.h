// Internal interface between the host side (products_host.cpp) and the kernels
// of the operators in opt8_products.h (fp8_quantize.hip, fp8_product.hip,
// gated_ffn.hip).  Not part of the public ABI.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

#include "../../include/opt8_products.h"
#include "products_choice.h"

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

}  // namespace opt8
