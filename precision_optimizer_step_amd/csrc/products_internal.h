// Internal interface between the host side (products_host.cpp) and the kernels
// of the operators in opt8_products.h (fp8_quantize.hip, fp8_product.hip,
// gated_ffn.hip).  Not part of the public ABI.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

#include "../../include/opt8_products.h"

namespace opt8 {

// Each queues its launches for validated, non-empty arguments.
hipError_t launch_fp8_quantize(const opt8_fp8_quant& q, hipStream_t stream);
hipError_t launch_fp8_matmul(const opt8_fp8_product& p, hipStream_t stream);
hipError_t launch_gated_ffn_forward(const opt8_gated_ffn& f, hipStream_t stream);
hipError_t launch_gated_ffn_backward(const opt8_gated_ffn_grad& g, hipStream_t stream);

// Rows of one of the two halves (dg, du) of the backward pass's workspace: f
// rounded up to whole steps of the contraction (64), the rest zeros.
inline int64_t gated_width(int64_t f) { return (f + 63) / 64 * 64; }
// Bytes of dg and du together.
inline int64_t gated_bytes(int64_t rows, int64_t f) { return rows * 2 * gated_width(f) * 2; }

}  // namespace opt8
