// 8 consecutive values of a row: loads, sums in 32 bits and stores, for the
// kernels whose lanes take a row in pieces of 8.
#pragma once

#include "tile_product.h"

namespace opt8 {
namespace tile {

template <class X> struct Raw { typedef uint16_t type; };
template <> struct Raw<float> { typedef float type; };

// 8 consecutive values as they lie in memory (16-bit ones stay packed until they
// are used: 32 registers for a thread's 64 values instead of 64); `left` of them
// exist, the others are zero.
template <class X>
struct Eight {
  i16x8 v;
  __device__ __forceinline__ void zero() { v = i16x8{0, 0, 0, 0, 0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const uint16_t* p, int64_t left) {
    if (left >= 8) {
      v = __builtin_bit_cast(i16x8, static_cast<i32x4>(*reinterpret_cast<const i32x4_at2*>(p)));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? static_cast<short>(p[i]) : 0;
    }
  }
  // The same for values that are read once, by a call too large for the caches to keep
  // any of it (streams() below): past them.
  __device__ __forceinline__ void stream(const uint16_t* p, int64_t left) {
    if (left >= 8) v = __builtin_bit_cast(i16x8, static_cast<i32x4>(__builtin_nontemporal_load(reinterpret_cast<const i32x4_at2*>(p))));
    else load(p, left);
  }
  __device__ __forceinline__ float operator[](int i) const { return value_of<X>(static_cast<uint16_t>(v[i])); }
};
template <>
struct Eight<float> {
  float v[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
  __device__ __forceinline__ void load(const float* p, int64_t left) {
    if (left >= 8) {
      const f32x4 a = *reinterpret_cast<const f32x4_at4*>(p), b = *reinterpret_cast<const f32x4_at4*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.0f;
    }
  }
  // (through the caches: a lane's 32 bytes are two loads, which share every line)
  __device__ __forceinline__ void stream(const float* p, int64_t left) { load(p, left); }
  __device__ __forceinline__ float operator[](int i) const { return v[i]; }
};

// The first `left` (at most 8) of 8 values, each rounded once to X.
template <class X>
__device__ __forceinline__ void store_eight(typename Raw<X>::type* p, const float* v, int64_t left) {
  if constexpr (sizeof(typename Raw<X>::type) == 4) store_some(p, v, left);
  else store_some(p, packed<X>(v), left);
}

// The same for results that leave in long streams: 16-bit ones are marked as not to be
// kept and leave the caches to what is read again.  16384 embeddings of 4096 bf16 values
// with places: 54.5 us without the mark, 38.8 with it; 2048: 7.2 and 6.9; 333: 2.9 both; norms
// with residual and codes 115 and 101, their backward pass 100.6 and 95.6, 64032 norms
// of 128 7.3 and 7.0.  32-bit ones are not: a lane's 32 bytes are two stores to a line,
// which meet in a cache (gradient of 50257 x 2048 fp32 embeddings: 147 us, with the mark
// 203).
template <class X>
__device__ __forceinline__ void stream_eight(typename Raw<X>::type* p, const float* v, int64_t left) {
  if constexpr (sizeof(typename Raw<X>::type) == 4) {
    store_some(p, v, left);
  } else {
    if (left < 8) store_some(p, packed<X>(v), left);
    else __builtin_nontemporal_store(packed<X>(v), reinterpret_cast<i32x4_at2*>(p));
  }
}

}  // namespace tile
}  // namespace opt8
