// Root-mean-square norm of rows, with the residual's addition and 8-bit codes, and
// its backward pass.
#include "fp8_codes.h"
#include "layers_internal.h"

namespace opt8 {
namespace {

using namespace tile;

// Sum over the 16 lanes of a row, in every one of them.
__device__ __forceinline__ float sum_of_16(float x) {
  x += rotated<0x121>(x);
  x += rotated<0x122>(x);
  x += rotated<0x124>(x);
  return x + rotated<0x128>(x);
}

__device__ __forceinline__ double sum_of_16(double x) {
  auto turned = [](double v, auto control) {
    const uint64_t bits = __builtin_bit_cast(uint64_t, v);
    const int low = __builtin_amdgcn_update_dpp(0, static_cast<int>(bits), decltype(control)::value, 0xf, 0xf, false);
    const int high = __builtin_amdgcn_update_dpp(0, static_cast<int>(bits >> 32), decltype(control)::value, 0xf, 0xf, false);
    return __builtin_bit_cast(double, static_cast<uint64_t>(static_cast<uint32_t>(high)) << 32 | static_cast<uint32_t>(low));
  };
  x += turned(x, std::integral_constant<int, 0x121>{});
  x += turned(x, std::integral_constant<int, 0x122>{});
  x += turned(x, std::integral_constant<int, 0x124>{});
  return x + turned(x, std::integral_constant<int, 0x128>{});
}

// Sum over the LANES lanes that share a row, in every one of them.  Where these are
// more than a wave, `slots` (one for each wave) carries the waves' sums; the caller
// alternates between two of them, so that one meeting of the waves is enough.
template <int LANES, class T>
__device__ __forceinline__ T sum_of(T x, T* slots) {
  x = sum_of_16(x);
  if constexpr (LANES > 16) {
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
  }
  if constexpr (LANES > 64) {
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = x;
    __syncthreads();
    x = slots[0];
#pragma unroll
    for (int w = 1; w < LANES / 64; ++w) x += slots[w];
  }
  return x;
}

// 8 weights, of the rows' type or of 32 bits.
template <class X>
__device__ __forceinline__ void load_weight(const void* weight, bool wide, int64_t c, int64_t left, float* w) {
  if (wide) {
    Eight<float> v;
    v.load(static_cast<const float*>(weight) + c, left);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i];
  } else {
    Eight<X> v;
    v.load(static_cast<const typename Raw<X>::type*>(weight) + c, left);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i];
  }
}

// ---------------------------------------------------------------- forward
struct Norm {
  const void* x;
  const void* residual;
  const void* weight;
  void* sum;
  void* y;
  uint8_t* q;
  float* scale;
  float* rstd;
  int64_t rows, d, ldx, ldresidual, ldsum, ldy, ldq;
  double eps, mean;   // mean: 1 / d
  int wide_weight, stream, stays;
};

// Squares are added up in 64 bits: no row of finite values is too large or too small for
// them, with an eps of 0 too, and rstd is rounded once.  A Newton step on the hardware's
// reciprocal root: 64032 norms of 128 in 7.0 us (32-bit sums 6.95; sqrt and a division in
// 64 bits 7.5), 16384 of 4096 in 100 either way.
__device__ __forceinline__ double add_squares(const float* t, double sum) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double v = static_cast<double>(t[i]);
    sum = __builtin_fma(v, v, sum);
  }
  return sum;
}
__device__ __forceinline__ float rstd_of(const Norm& p, double squares) {
  const double m = squares * p.mean + p.eps, y = __builtin_amdgcn_rsq(m);    // to about 2^-24
  const double rest = __builtin_fma(-(m * y), y, 1.0);                       // NaN where m is 0 or infinite: y is the answer
  return static_cast<float>(rest == rest ? __builtin_fma(0.5 * y, rest, y) : y);
}

// t of 8 columns, and its place in `sum`.
template <class X>
__device__ __forceinline__ void residual_sum(const Norm& p, const Eight<X>& x, const Eight<X>& r, float* t) {
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = p.residual ? x[i] + r[i] : x[i];
}

// The outputs of 8 columns but `sum`, from t; all 16 lanes of a block call it.
template <class X, int F>
__device__ __forceinline__ void norm_out(const Norm& p, int64_t row, int64_t c, int64_t left, float rstd, const float* t, const float* w) {
  float n[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) n[i] = (t[i] * rstd) * w[i];
  if (p.y && left > 0) {
    auto* to = static_cast<typename Raw<X>::type*>(p.y) + row * p.ldy + c;
    if (p.stays) store_eight<X>(to, n, left);
    else stream_eight<X>(to, n, left);
  }
  if constexpr (F >= 0) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = larger(top, n[i]);
    const float s = scale_of<F>(largest_of_16(top));
    const float inv = 1.0f / s;
    if (left > 0) {
      if ((threadIdx.x & 15) == 0) p.scale[(c >> 7) * p.rows + row] = s;
      const uint32_t a = code4<F>(n[0] * inv, n[1] * inv, n[2] * inv, n[3] * inv);
      const uint32_t b = code4<F>(n[4] * inv, n[5] * inv, n[6] * inv, n[7] * inv);
      uint8_t* o = p.q + row * p.ldq + c;
      if (left >= 8) {
        *reinterpret_cast<uint2*>(o) = uint2{a, b};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < left) o[i] = static_cast<uint8_t>((i < 4 ? a : b) >> (8 * (i & 3)));
      }
    }
  }
}

// LANES lanes share a row and hold it in K pieces of 8 columns each, so that it is
// read once.  F: codes of e4m3 (0), e5m2 (1) or none (-1).  Bound by memory: 16384 x 4096
// bf16 with residual, y and codes 100 us, 604 MB (6.0 TB/s).  Workgroups take the rows in
// their order: with a run of neighbouring rows to each XCD 117 us (the lines of scales,
// which 32 neighbouring rows share, would meet in one L2; as it is 16 MB more are written
// than needed).  A wave to such a row, without a meeting of waves, 125.  16384 columns:
// 512 lanes 117 us, 256 with twice the registers 126-132.
template <class X, int F, int LANES, int K>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256) void norm_kernel(const Norm p) {
  constexpr int kRows = LANES > 256 ? 1 : 256 / LANES;    // to a workgroup
  __shared__ double slots[16];
  typedef typename Raw<X>::type Value;
  const int l = threadIdx.x % LANES;
  const int64_t row = int64_t{blockIdx.x} * kRows + threadIdx.x / LANES;
  const bool there = row < p.rows;
  Eight<X> x[K], r[K];
  float w[K][8], t[K][8];
  auto read = [&](auto&& one) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t c = (k * LANES + l) * 8, left = there ? p.d - c : 0;
      x[k].zero();
      r[k].zero();
      if (left > 0) {
        one(x[k], static_cast<const Value*>(p.x) + row * p.ldx + c, left);
        if (p.residual) one(r[k], static_cast<const Value*>(p.residual) + row * p.ldresidual + c, left);
      }
    }
  };
  if (p.stream) read([](Eight<X>& v, const Value* at, int64_t left) { v.stream(at, left); });
  else read([](Eight<X>& v, const Value* at, int64_t left) { v.load(at, left); });
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t c = (k * LANES + l) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[k][i] = 0.0f;
    if (c < p.d) load_weight<X>(p.weight, p.wide_weight, c, p.d - c, w[k]);
  }
  double squares = 0.0;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t c = (k * LANES + l) * 8, left = there ? p.d - c : 0;
    residual_sum<X>(p, x[k], r[k], t[k]);
    if (p.sum && left > 0) stream_eight<X>(static_cast<Value*>(p.sum) + row * p.ldsum + c, t[k], left);
    squares = add_squares(t[k], squares);
  }
  const float rstd = rstd_of(p, sum_of<LANES>(squares, slots));
  if (p.rstd && there && l == 0) p.rstd[row] = rstd;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t c = (k * LANES + l) * 8;
    norm_out<X, F>(p, row, c, there ? p.d - c : 0, rstd, t[k], w[k]);
  }
}

// Longer rows are read twice, by a workgroup each: 3000 x 20000 bf16 with residual, y and
// codes 120 us, 782 MB with the second reading (6.5 TB/s, part of it from the caches); fp32
// without residual 112.
template <class X, int F>
__global__ __launch_bounds__(1024) void norm_long_kernel(const Norm p) {
  __shared__ double slots[16];
  typedef typename Raw<X>::type Value;
  const int64_t row = blockIdx.x;
  const Value* xs = static_cast<const Value*>(p.x) + row * p.ldx;
  const Value* rs = static_cast<const Value*>(p.residual) + (p.residual ? row * p.ldresidual : 0);
  double squares = 0.0;
  for (int64_t c = threadIdx.x * 8; c < p.d; c += 8192) {
    Eight<X> x, r;
    float t[8];
    r.zero();
    x.load(xs + c, p.d - c);
    if (p.residual) r.load(rs + c, p.d - c);
    residual_sum<X>(p, x, r, t);
    squares = add_squares(t, squares);
  }
  const float rstd = rstd_of(p, sum_of<1024>(squares, slots));
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  for (int64_t c0 = 0; c0 < p.d; c0 += 8192) {    // all lanes of a block stay in the loop
    const int64_t c = c0 + threadIdx.x * 8, left = p.d - c;
    Eight<X> x, r;
    float t[8], w[8] = {};
    x.zero();
    r.zero();
    if (left > 0) {
      x.load(xs + c, left);
      if (p.residual) r.load(rs + c, left);
      load_weight<X>(p.weight, p.wide_weight, c, left, w);
    }
    residual_sum<X>(p, x, r, t);
    if (p.sum && left > 0) stream_eight<X>(static_cast<Value*>(p.sum) + row * p.ldsum + c, t, left);
    norm_out<X, F>(p, row, c, left, rstd, t, w);
  }
}

template <class X, int F, int LANES, int K>
hipError_t launch_held(Norm& p, hipStream_t stream) {
  constexpr int kThreads = LANES > 256 ? LANES : 256;
  return queue(norm_kernel<X, F, LANES, K>, static_cast<unsigned>(pieces_of(p.rows, kThreads / LANES)), kThreads, stream, p);
}

template <class X, int F>
hipError_t launch_norm(Norm& p, hipStream_t stream) {
  if (p.d <= 128) return launch_held<X, F, 16, 1>(p, stream);
  if (p.d <= 512) return launch_held<X, F, 64, 1>(p, stream);
  if (p.d <= 1024) return launch_held<X, F, 64, 2>(p, stream);
  if (p.d <= 2048) return launch_held<X, F, 256, 1>(p, stream);
  if (p.d <= 4096) return launch_held<X, F, 256, 2>(p, stream);
  if (p.d <= 8192) return launch_held<X, F, 256, 4>(p, stream);
  if (p.d <= kNormHeld) return launch_held<X, F, 512, 4>(p, stream);
  return queue(norm_long_kernel<X, F>, static_cast<unsigned>(p.rows), 1024, stream, p);
}

template <class X>
hipError_t launch_codes(Norm& p, int q_type, hipStream_t stream) {
  if (!p.q) return launch_norm<X, -1>(p, stream);
  return q_type == OPT8_TYPE_E4M3 ? launch_norm<X, 0>(p, stream) : launch_norm<X, 1>(p, stream);
}

// ---------------------------------------------------------------- backward
struct NormGrad {
  const void* dy;
  const void* x;
  const void* weight;
  const float* rstd;
  const void* dsum;
  void* dx;
  void* dweight;     // with one group
  float* partial;    // [groups][d] with more, or NULL where there is no dweight
  int64_t rows, d, lddy, ldx, lddsum, lddx;
  int groups;
  float mean;
  int wide_weight, wide_dweight, stream;
};

// Sums of dweight's columns, rounded (a lone workgroup) or left to the second kernel.
template <class X>
__device__ __forceinline__ void give_dweight(const NormGrad& p, int64_t c, const float* sum) {
  const int64_t left = p.d - c;
  if (left <= 0) return;
  if (p.groups > 1) store_some(p.partial + blockIdx.x * p.d + c, sum, left);
  else if (p.wide_dweight) store_some(static_cast<float*>(p.dweight) + c, sum, left);
  else store_eight<X>(static_cast<typename Raw<X>::type*>(p.dweight) + c, sum, left);
}

// As norm_kernel, but a workgroup walks through the rows, every p.groups-th of them
// (or of their groups), and keeps its sums of dweight in registers; the next row is
// on its way while one is computed.  Bound by memory: 16384 x 4096 bf16 with dsum 89-93
// us, 546 MB (6 TB/s).  The widest form (over 8192 columns) spills registers, 84 bytes of a
// lane with 16-bit rows: 4096 x 16384 122 us for the same bytes.  Few or short rows are
// bound by the bytes under way, a row (or 16 short ones) to a workgroup at a time, 13 to 16
// KB to a CU: 4001 x 1600 fp16 38 MB in 12.8 us, 64032 x 128 49 MB in 12 (3 and 4 TB/s).
template <class X, int LANES, int K>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256) void norm_grad_kernel(const NormGrad p) {
  constexpr int kThreads = LANES > 256 ? LANES : 256, kRows = kThreads / LANES;
  typedef typename Raw<X>::type Value;
  __shared__ float slots[2][16];
  __shared__ float joined[kRows > 1 ? kRows : 1][kRows > 1 ? LANES * K * 8 : 1];
  const int l = threadIdx.x % LANES, g = threadIdx.x / LANES;
  float w[K][8], sums[K][8] = {};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t c = (k * LANES + l) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[k][i] = 0.0f;
    if (p.dx && c < p.d) load_weight<X>(p.weight, p.wide_weight, c, p.d - c, w[k]);
  }
  Eight<X> dy[K], x[K], ds[K];
  float rstd = 0.0f;
  const int64_t step = int64_t{p.groups} * kRows;
  auto read = [&](int64_t row, auto&& one) {
    const bool there = row < p.rows;
    rstd = there ? p.rstd[row] : 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t c = (k * LANES + l) * 8, left = there ? p.d - c : 0;
      dy[k].zero();
      x[k].zero();
      ds[k].zero();
      if (left > 0) {
        one(dy[k], static_cast<const Value*>(p.dy) + row * p.lddy + c, left);
        one(x[k], static_cast<const Value*>(p.x) + row * p.ldx + c, left);
        if (p.dsum) one(ds[k], static_cast<const Value*>(p.dsum) + row * p.lddsum + c, left);
      }
    }
  };
  auto load = [&](int64_t row) {
    if (p.stream) read(row, [](Eight<X>& v, const Value* at, int64_t left) { v.stream(at, left); });
    else read(row, [](Eight<X>& v, const Value* at, int64_t left) { v.load(at, left); });
  };
  load(int64_t{blockIdx.x} * kRows + g);
  int turn = 0;
  for (int64_t r0 = int64_t{blockIdx.x} * kRows; r0 < p.rows; r0 += step) {
    const int64_t row = r0 + g;
    const float at = rstd;
    float a[K][8], h[K][8], more[K][8], along = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[k][i] = x[k][i] * at;
        const float v = dy[k][i];
        sums[k][i] = __builtin_fmaf(v, h[k][i], sums[k][i]);
        a[k][i] = v * w[k][i];
        along = __builtin_fmaf(a[k][i], h[k][i], along);
        more[k][i] = ds[k][i];
      }
    load(row + step);
    if (p.dx) {
      along = sum_of<LANES>(along, slots[turn]) * p.mean;
      turn ^= 1;
      if (row < p.rows)
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int64_t c = (k * LANES + l) * 8, left = p.d - c;
          if (left <= 0) continue;
          float out[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            out[i] = at * __builtin_fmaf(-along, h[k][i], a[k][i]);
            if (p.dsum) out[i] += more[k][i];
          }
          stream_eight<X>(static_cast<Value*>(p.dx) + row * p.lddx + c, out, left);
        }
    }
  }
  if (!p.dweight) return;
  if constexpr (kRows > 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) joined[g][(k * LANES + l) * 8 + i] = sums[k][i];
    __syncthreads();
    for (int c = threadIdx.x * 8; c < LANES * K * 8; c += kThreads * 8) {
      float sum[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[i] = joined[0][c + i];
#pragma unroll
        for (int r = 1; r < kRows; ++r) sum[i] += joined[r][c + i];
      }
      give_dweight<X>(p, c, sum);
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) give_dweight<X>(p, (k * LANES + l) * 8, sums[k]);
  }
}

// Rows too long to be held: sums of dweight by columns, a thread 8 of them over every
// p.groups-th row.  With dx below, dy and x are read three times: 3000 x 20000 bf16 with dsum
// 155 us, 50 of them here.
template <class X>
__global__ __launch_bounds__(256) void dweight_long_kernel(const NormGrad p) {
  typedef typename Raw<X>::type Value;
  const int64_t blocks = (p.d + 2047) / 2048;
  const int64_t c = blockIdx.x % blocks * 2048 + threadIdx.x * 8, left = p.d - c;
  const int64_t group = blockIdx.x / blocks;
  if (left <= 0) return;
  float sums[8] = {};
#pragma unroll 4
  for (int64_t row = group; row < p.rows; row += p.groups) {
    Eight<X> dy, x;
    dy.load(static_cast<const Value*>(p.dy) + row * p.lddy + c, left);
    x.load(static_cast<const Value*>(p.x) + row * p.ldx + c, left);
    const float rstd = p.rstd[row];
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[i] = __builtin_fmaf(dy[i], x[i] * rstd, sums[i]);
  }
  store_some(p.partial + group * p.d + c, sums, left);
}

template <class X>
__global__ __launch_bounds__(1024) void dx_long_kernel(const NormGrad p) {
  typedef typename Raw<X>::type Value;
  __shared__ float slots[16];
  const int64_t row = blockIdx.x;
  const Value* dys = static_cast<const Value*>(p.dy) + row * p.lddy;
  const Value* xs = static_cast<const Value*>(p.x) + row * p.ldx;
  const float rstd = p.rstd[row];
  float along = 0.0f;
  for (int64_t c = threadIdx.x * 8; c < p.d; c += 8192) {
    Eight<X> dy, x;
    float w[8];
    dy.load(dys + c, p.d - c);
    x.load(xs + c, p.d - c);
    load_weight<X>(p.weight, p.wide_weight, c, p.d - c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) along = __builtin_fmaf(dy[i] * w[i], x[i] * rstd, along);
  }
  along = sum_of<1024>(along, slots) * p.mean;
  for (int64_t c = threadIdx.x * 8; c < p.d; c += 8192) {
    Eight<X> dy, x, ds;
    float w[8], out[8];
    dy.load(dys + c, p.d - c);
    x.load(xs + c, p.d - c);
    ds.zero();
    if (p.dsum) ds.load(static_cast<const Value*>(p.dsum) + row * p.lddsum + c, p.d - c);
    load_weight<X>(p.weight, p.wide_weight, c, p.d - c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      out[i] = rstd * __builtin_fmaf(-along, x[i] * rstd, dy[i] * w[i]);
      if (p.dsum) out[i] += ds[i];
    }
    stream_eight<X>(static_cast<Value*>(p.dx) + row * p.lddx + c, out, p.d - c);
  }
}

// dweight from the workgroups' sums: a workgroup takes 32 columns, 4 to a lane, and 128
// lanes an equal share of the sums each, whose joint sums meet in LDS.  With no rows
// (no groups) it stores zeros.  512 sums of 4096 columns: 4.5 us.
template <class D>
__global__ __launch_bounds__(1024) void dweight_kernel(const NormGrad p) {
  __shared__ f32x4 parts[128][9];
  const int t = threadIdx.x, l = t & 7, slot = t >> 3;
  const int64_t c = int64_t{blockIdx.x} * 32 + l * 4;
  const int left = static_cast<int>(p.d - c < 4 ? p.d - c : 4);
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int g = slot; g < p.groups; g += 128) {
    const float* at = p.partial + int64_t{g} * p.d + c;
    if (left == 4) {
      sum += *reinterpret_cast<const f32x4_at4*>(at);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) sum[i] += at[i];
    }
  }
  parts[slot][l] = sum;
  for (int half = 64; half > 0; half >>= 1) {
    __syncthreads();
    if (slot < half) parts[slot][l] += parts[slot + half][l];
  }
  if (slot > 0 || left <= 0) return;
  sum = parts[0][l];
  auto* out = static_cast<typename Raw<D>::type*>(p.dweight) + c;
  for (int i = 0; i < left; ++i) {
    if constexpr (sizeof(typename Raw<D>::type) == 4) out[i] = sum[i];
    else out[i] = static_cast<uint16_t>(bits_of(D{}, sum[i]));
  }
}

template <class X>
hipError_t launch_grad(NormGrad& p, hipStream_t stream) {
  hipError_t e = hipSuccess;
  const unsigned groups = static_cast<unsigned>(p.groups);
  if (p.rows == 0) {
    p.groups = 0;
  } else if (p.d <= kNormHeld) {
    const RowShape shape = norm_grad_shape(p.d);
    if (shape.lanes == 16) e = queue(norm_grad_kernel<X, 16, 1>, groups, 256, stream, p);
    else if (shape.lanes == 64 && shape.pieces == 1) e = queue(norm_grad_kernel<X, 64, 1>, groups, 256, stream, p);
    else if (shape.lanes == 64) e = queue(norm_grad_kernel<X, 64, 2>, groups, 256, stream, p);
    else if (shape.lanes == 256 && shape.pieces == 1) e = queue(norm_grad_kernel<X, 256, 1>, groups, 256, stream, p);
    else if (shape.lanes == 256) e = queue(norm_grad_kernel<X, 256, 2>, groups, 256, stream, p);
    else if (shape.pieces == 1) e = queue(norm_grad_kernel<X, 1024, 1>, groups, 1024, stream, p);
    else e = queue(norm_grad_kernel<X, 1024, 2>, groups, 1024, stream, p);
    if (p.groups == 1) return e;
  } else {
    // dweight first: dx may take dy's place
    if (p.dweight) e = queue(dweight_long_kernel<X>, static_cast<unsigned>(p.groups * pieces_of(p.d, 2048)), 256, stream, p);
    if (e == hipSuccess && p.dx) e = queue(dx_long_kernel<X>, static_cast<unsigned>(p.rows), 1024, stream, p);
  }
  if (e != hipSuccess || !p.dweight) return e;
  const unsigned blocks = static_cast<unsigned>(pieces_of(p.d, 32));
  return p.wide_dweight ? queue(dweight_kernel<float>, blocks, 1024, stream, p) : queue(dweight_kernel<X>, blocks, 1024, stream, p);
}

}  // namespace

hipError_t launch_rms_norm_forward(const opt8_rms_norm& a, hipStream_t stream) {
  Norm p;
  p.x = a.x;
  p.residual = a.residual;
  p.weight = a.weight;
  p.sum = a.sum;
  p.y = a.y;
  p.q = static_cast<uint8_t*>(a.q);
  p.scale = a.scale;
  p.rstd = a.rstd;
  p.rows = a.rows;
  p.d = a.d;
  p.ldx = a.ldx;
  p.ldresidual = a.ldresidual;
  p.ldsum = a.ldsum;
  p.ldy = a.ldy;
  p.ldq = a.ldq;
  p.eps = a.eps;
  p.mean = 1.0 / static_cast<double>(a.d);
  p.wide_weight = a.weight_type == OPT8_TYPE_FP32 && a.type != OPT8_TYPE_FP32;
  p.stream = streams(a.rows * a.d * (a.residual ? 6 : 4));
  p.stays = stays(a.rows * a.d * 2);
  if (a.type == OPT8_TYPE_BF16) return launch_codes<Bf16>(p, a.q_type, stream);
  if (a.type == OPT8_TYPE_FP16) return launch_codes<Fp16>(p, a.q_type, stream);
  return launch_codes<float>(p, a.q_type, stream);
}

hipError_t launch_rms_norm_backward(const opt8_rms_norm_grad& a, hipStream_t stream) {
  NormGrad p;
  p.dy = a.dy;
  p.x = a.x;
  p.weight = a.weight;
  p.rstd = a.rstd;
  p.dsum = a.dsum;
  p.dx = a.dx;
  p.dweight = a.dweight;
  p.partial = static_cast<float*>(a.workspace);
  p.rows = a.rows;
  p.d = a.d;
  p.lddy = a.lddy;
  p.ldx = a.ldx;
  p.lddsum = a.lddsum;
  p.lddx = a.lddx;
  p.groups = static_cast<int>(norm_grad_groups(a.rows, a.d));
  p.mean = static_cast<float>(1.0 / static_cast<double>(a.d));
  p.wide_weight = a.weight_type == OPT8_TYPE_FP32 && a.type != OPT8_TYPE_FP32;
  p.wide_dweight = a.dweight_type == OPT8_TYPE_FP32 && a.type != OPT8_TYPE_FP32;
  p.stream = streams(a.rows * a.d * (a.dsum ? 8 : 6));
  if (a.type == OPT8_TYPE_BF16) return launch_grad<Bf16>(p, stream);
  if (a.type == OPT8_TYPE_FP16) return launch_grad<Fp16>(p, stream);
  return launch_grad<float>(p, stream);
}

}  // namespace opt8
