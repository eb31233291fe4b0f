// Internal interface between the host side (layers_host.cpp) and the kernels of
// the operators in opt8_layers.h (embedding.hip, rms_norm.hip, grad_norm.hip).
// Not part of the public ABI.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

#include "../../include/opt8_layers.h"
#include "layers_sizes.h"
#include "products_internal.h"

namespace opt8 {

// One piece of a gradient of a list, as opt8_grad_table writes it.
struct GradPiece {
  const void* from;
  void* to;
  int32_t count;
  int16_t type, to_type;
};
static_assert(sizeof(GradPiece) == OPT8_GRAD_PIECE_BYTES, "the table's layout");

// What stands before the pieces in a table.
struct GradHead {
  int64_t pieces;
  int64_t own;       // of them with a place of their own for what is clipped: the first ones
  int64_t reserved;
};
static_assert(sizeof(GradHead) == OPT8_GRAD_PIECE_BYTES, "the table's layout");

// Each queues its launches for validated, non-empty arguments.
hipError_t launch_embedding_forward(const opt8_embedding& a, hipStream_t stream);
hipError_t launch_embedding_backward(const opt8_embedding_grad& a, hipStream_t stream);
hipError_t launch_rms_norm_forward(const opt8_rms_norm& a, hipStream_t stream);
hipError_t launch_rms_norm_backward(const opt8_rms_norm_grad& a, hipStream_t stream);
hipError_t launch_grad_norm(const opt8_grads& a, hipStream_t stream);
hipError_t launch_grad_clip(const opt8_grads& a, hipStream_t stream);

}  // namespace opt8
