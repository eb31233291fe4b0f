// 8-bit codes and the scales of blocks of 128 values, for kernels whose 16
// adjacent lanes hold a block.
#pragma once

#include "vectors.h"

namespace opt8 {
namespace tile {

// The largest of the 16 lanes of a row, in every one of them: rotations by 1, 2,
// 4 and 8 lanes.
template <int CONTROL>
__device__ __forceinline__ float rotated(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CONTROL, 0xf, 0xf, false));
}
__device__ __forceinline__ float largest_of_16(float x) {
  x = __builtin_fmaxf(x, rotated<0x121>(x));
  x = __builtin_fmaxf(x, rotated<0x122>(x));
  x = __builtin_fmaxf(x, rotated<0x124>(x));
  return __builtin_fmaxf(x, rotated<0x128>(x));
}

// The largest magnitude so far; NaN does not count (fmaxf returns the other).
__device__ __forceinline__ float larger(float top, float x) { return __builtin_fmaxf(top, __builtin_fabsf(x)); }

template <int F> constexpr float kLargest = F == 0 ? 448.0f : 57344.0f;
template <int F>
__device__ __forceinline__ float scale_of(float top) { return __builtin_fmaxf(top / kLargest<F>, 0x1p-126f); }

// Codes of four values.  No product passes the largest value by more than its
// own rounding, so the conversion cannot overflow.
template <int F>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
  int w = 0;
  if constexpr (F == 0) {
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  } else {
    w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
  }
  return static_cast<uint32_t>(w);
}

}  // namespace tile
}  // namespace opt8
