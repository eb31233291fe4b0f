// 8-bit codes and block scales of a matrix, of its transpose, or of both from
// one read of it.
#include <algorithm>

#include "fp8_codes.h"
#include "products_internal.h"

namespace opt8 {
namespace {

using namespace tile;

struct Quant {
  const void* x;
  uint8_t* q;
  float* scale;
  uint8_t* qt;
  float* scale_t;
  int64_t rows, cols, ldx, ldq, ldt;
  int cb, rb;    // blocks of columns and of rows
};

// A workgroup takes one 128 x 128 tile: thread t holds the 8 x 8 values of
// rows 8*(t/16).. and columns 8*(t%16).. in registers, so x is read once for
// both orientations.  A row's maximum is reduced over its 16 lanes, a column's
// over the 16 row groups through LDS.  The transposed codes leave as 8-byte
// runs of a column, four lanes of a wave side by side.  Bound by memory: 16384 x
// 4096 bf16 by tiles, both ways, 62 us (4.3 TB/s); 4001 x 10240 by rows, both ways,
// 44 us (3.8 TB/s); 48 and 33 us where the last call's data, the same, are still in the
// last-level cache.
template <class X, int F, bool TILE, bool Q, bool T>
__global__ __launch_bounds__(256) void quantize_kernel(const Quant p) {
  __shared__ float tops[16][128];
  __shared__ float wave_top[4];
  const int t = threadIdx.x, lane16 = t & 15, rg = t >> 4;
  const int cblk = blockIdx.x % p.cb, rblk = blockIdx.x / p.cb;
  const int64_t r0 = int64_t{rblk} * 128 + rg * 8, c0 = int64_t{cblk} * 128 + lane16 * 8;
  const auto* x = static_cast<const typename Raw<X>::type*>(p.x);
  Eight<X> v[8];
  const int64_t cleft = p.cols - c0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + i < p.rows && cleft > 0) v[i].load(x + (r0 + i) * p.ldx + c0, cleft);
    else v[i].zero();
  }

  float inv[8], invt[8];
  if constexpr (TILE) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) top = larger(top, v[i][j]);
    top = largest_of_16(top);
    top = __builtin_fmaxf(top, __shfl_xor(top, 16));
    top = __builtin_fmaxf(top, __shfl_xor(top, 32));
    if ((t & 63) == 0) wave_top[t >> 6] = top;
    __syncthreads();
    top = __builtin_fmaxf(__builtin_fmaxf(wave_top[0], wave_top[1]), __builtin_fmaxf(wave_top[2], wave_top[3]));
    const float s = scale_of<F>(top);
    if (t == 0) {
      if constexpr (Q) p.scale[int64_t{cblk} * p.rb + rblk] = s;
      if constexpr (T) p.scale_t[int64_t{rblk} * p.cb + cblk] = s;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) inv[i] = invt[i] = 1.0f / s;
  } else {
    if constexpr (Q) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = larger(top, v[i][j]);
        const float s = scale_of<F>(largest_of_16(top));
        inv[i] = 1.0f / s;
        if (lane16 == i && r0 + i < p.rows) p.scale[int64_t{cblk} * p.rows + r0 + i] = s;
      }
    }
    if constexpr (T) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = larger(top, v[i][j]);
        tops[rg][lane16 * 8 + j] = top;
      }
      __syncthreads();
      if (t < 128) {
        float top = tops[0][t];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = __builtin_fmaxf(top, tops[i][t]);
        const float s = scale_of<F>(top);
        const int64_t c = int64_t{cblk} * 128 + t;
        if (c < p.cols) p.scale_t[int64_t{rblk} * p.cols + c] = s;
        tops[0][t] = 1.0f / s;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) invt[j] = tops[0][lane16 * 8 + j];
    }
  }

  if constexpr (Q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i >= p.rows || cleft <= 0) continue;
      uint32_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[h] = code4<F>(v[i][4 * h] * inv[i], v[i][4 * h + 1] * inv[i], v[i][4 * h + 2] * inv[i], v[i][4 * h + 3] * inv[i]);
      uint8_t* o = p.q + (r0 + i) * p.ldq + c0;
      if (cleft >= 8) {
        *reinterpret_cast<uint2*>(o) = uint2{w[0], w[1]};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < cleft) o[j] = static_cast<uint8_t>(w[j >> 2] >> (8 * (j & 3)));
      }
    }
  }
  if constexpr (T) {
    const int64_t rleft = p.rows - r0;
    if (rleft > 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= cleft) continue;
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = code4<F>(v[4 * h][j] * invt[j], v[4 * h + 1][j] * invt[j], v[4 * h + 2][j] * invt[j], v[4 * h + 3][j] * invt[j]);
        uint8_t* o = p.qt + (c0 + j) * p.ldt + r0;
        if (rleft >= 8) {
          *reinterpret_cast<uint2*>(o) = uint2{w[0], w[1]};
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < rleft) o[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
        }
      }
    }
  }
}

template <class X, int F, bool TILE>
hipError_t launch(Quant& p, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(int64_t{p.cb} * p.rb);
  if (p.q && p.qt) return queue(quantize_kernel<X, F, TILE, true, true>, grid, 256, stream, p);
  if (p.q) return queue(quantize_kernel<X, F, TILE, true, false>, grid, 256, stream, p);
  return queue(quantize_kernel<X, F, TILE, false, true>, grid, 256, stream, p);
}

template <class X>
hipError_t launch_format(Quant& p, int format, int block, hipStream_t stream) {
  if (format == OPT8_TYPE_E4M3)
    return block == OPT8_FP8_BLOCK_TILE ? launch<X, 0, true>(p, stream) : launch<X, 0, false>(p, stream);
  return block == OPT8_FP8_BLOCK_TILE ? launch<X, 1, true>(p, stream) : launch<X, 1, false>(p, stream);
}

}  // namespace

hipError_t launch_fp8_quantize(const opt8_fp8_quant& a, hipStream_t stream) {
  Quant p;
  p.x = a.x;
  p.q = static_cast<uint8_t*>(a.q);
  p.scale = a.scale;
  p.qt = static_cast<uint8_t*>(a.qt);
  p.scale_t = a.scale_t;
  p.rows = a.rows;
  p.cols = a.cols;
  p.ldx = a.ldx;
  p.ldq = a.ldq;
  p.ldt = a.ldt;
  p.cb = static_cast<int>((a.cols + 127) / 128);
  p.rb = static_cast<int>((a.rows + 127) / 128);
  if (a.x_type == OPT8_TYPE_BF16) return launch_format<Bf16>(p, a.q_type, a.block, stream);
  if (a.x_type == OPT8_TYPE_FP16) return launch_format<Fp16>(p, a.q_type, a.block, stream);
  return launch_format<float>(p, a.q_type, a.block, stream);
}

}  // namespace opt8
