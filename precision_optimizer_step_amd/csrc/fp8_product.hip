// C = A B^T on 8-bit floating point operands with a scale for each 128 values of
// k: C[m][n] = sum_b (sa[b][m] * sb[b][n]) * sum_{k in b} A[m][k] B[n][k].
//
// Precision.  The 8-bit matrix instruction aligns each 8 products to the largest
// one and drops what lies 2^-13 below its power of two (measured: a term 2^-14 of
// another among the same 8 consecutive k is lost whole, in another 8 kept);
// sums of the 8s are fp32.  On normal values that is 1.5e-5 of the result in
// norm, a hundredth of bf16's rounding and a tenth of fp16's.
#include <algorithm>
#include <cstdint>

#include "products_internal.h"
#include "tile_product.h"

namespace opt8 {
namespace {

using namespace tile;

struct Product {
  const char* a;
  const float* sa;
  const char* b;
  const float* sb;
  uint16_t* c;
  int64_t lda, ldb, ldc;
  int m, n, k;
  int nb;        // entries of sb for one block of k
  int tiles_m, tiles_n, band;
  bool vec;      // C takes 16-byte stores
};

// (The body is for the device pass alone: the host pass of this compiler
// otherwise leaves out the launch stubs of some instances.)
//
// One BM x BN tile of C, WM x WN waves.  The scales of a step's block of k lie
// in LDS beside its operand tiles, one for each row of either (TILE scales are
// spread over their rows by the loads' addresses).
template <int FA, class C, bool TILE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void product_kernel(const Product p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = WM * WN;
  constexpr int MT = BM / WM / 16;
  static_assert(BN / WN == 64, "a wave takes 64 columns");
  static_assert((BM + BN) / 64 <= NW, "a wave loads at most 64 scales a step");
  constexpr int kTile = (BM + BN) * kStepBytes;
  __shared__ __align__(16) char lds[2][kTile + (BM + BN) * 4];

  int tm, tn;
  tile_of_group(p.tiles_m, p.tiles_n, p.band, tm, tn);
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int m0 = tm * BM, n0 = tn * BN;
  const int64_t kbytes = p.k, kround = (kbytes + 15) & ~int64_t{15};

  Loader<kRows, BM, NW> la;
  Loader<kRows, BN, NW> lb;
  la.init(p.a + m0 * p.lda, p.lda, (std::min(BM, p.m - m0) - 1) * p.lda + kround, 0, wave);
  lb.init(p.b + n0 * p.ldb, p.ldb, (std::min(BN, p.n - n0) - 1) * p.ldb + kround, 0, wave);
  const int steps = (p.k + kStepBytes - 1) / kStepBytes;

  // this wave's 64 scales: of A's rows (waves 0 .. BM/64 - 1) or of B's
  const bool scales_a = wave < BM / 64;
  const bool scales = wave < (BM + BN) / 64;
  const int srow = scales_a ? m0 + wave * 64 + lane : n0 + (wave - BM / 64) * 64 + lane;
  const int64_t sstep = scales_a ? p.m : p.nb;
  const char* sbase = reinterpret_cast<const char*>(scales_a ? p.sa : p.sb);
  uint32_t soff = static_cast<uint32_t>((scales_a || !TILE) ? srow : srow / 128) * 4;
  if (srow >= (scales_a ? p.m : p.n)) soff = kOutOfRange;

  auto issue = [&](int step) {
    char* to = lds[step & 1];
    la.at_step(step, p.k - step * kStepBytes);
    lb.at_step(step, p.k - step * kStepBytes);
#pragma unroll
    for (int j = 0; j < BM / 8 / NW; ++j) la.issue(lds_address(to), j);
#pragma unroll
    for (int j = 0; j < BN / 8 / NW; ++j) lb.issue(lds_address(to + BM * kStepBytes), j);
    if (scales)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(sbase + step * sstep * 4, sstep * 4),
                                               (lds_void*)(to + kTile + wave * 256), 4, soff, 0, 0, 0);
  };

  Reader<kRows, BM, MT / 2> ra;
  Reader<kRows, BN, 2> rb;
  ra.init(wm * (BM / WM));
  rb.init(wn * 64);
  const int mlane = 8 * ((lane & 15) >> 2) + (lane & 3);
  f32x4 acc[4][MT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  if (steps > 0) issue(0);
  for (int step = 0; step < steps; ++step) {
    wait_and_meet();
    if (step + 1 < steps) issue(step + 1);
    char* t = lds[step & 1];
    if (step + 1 == steps && (p.k & 15)) {
      clear_part_chunk<BM, 64 * NW>(t, p.k - step * kStepBytes);
      clear_part_chunk<BN, 64 * NW>(t + BM * kStepBytes, p.k - step * kStepBytes);
      __syncthreads();
    }
    const float* sa = reinterpret_cast<const float*>(t + kTile) + wm * (BM / WM);
    const float* sb = reinterpret_cast<const float*>(t + kTile) + BM + wn * 64;
    i32x8 b[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const i32x4 lo = rb.read(t + BM * kStepBytes, q, 0), hi = rb.read(t + BM * kStepBytes, q, 1);
      b[q] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    f32x4 sn[4];
    float s1 = 0;
    if constexpr (TILE) {
      s1 = sb[0];
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sn[q] = *reinterpret_cast<const f32x4*>(sb + (q >> 1) * 32 + 8 * (lane >> 4) + 4 * (q & 1));
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const i32x4 lo = ra.read(t, j, 0), hi = ra.read(t, j, 1);
      const i32x8 a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      float s = sa[(j >> 1) * 32 + 4 * (j & 1) + mlane];
      if constexpr (TILE) s *= s1;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 part = mfma8<FA>(b[q], a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = TILE ? s : s * sn[q][i];
          acc[q][j][i] = __builtin_fmaf(part[i], w, acc[q][j][i]);
        }
      }
    }
  }

#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int m = m0 + wm * (BM / WM) + (j >> 1) * 32 + 4 * (j & 1) + mlane;
    if (m >= p.m) continue;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int n = n0 + wn * 64 + q * 32 + 8 * (lane >> 4);
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = acc[2 * q][j][i];
        v[4 + i] = acc[2 * q + 1][j][i];
      }
      store8<C>(p.c + m * p.ldc + n, v, p.n - n, p.vec);
    }
  }
#endif
}

// Few rows (one token to a short prompt): the time is that of reading B, so
// nothing goes through LDS.  A workgroup owns 16 n and 16*MT m; its 4 waves
// take every fourth block of k, hold B's and A's fragments in registers straight
// from memory (a lane 32 bytes of a row's 128) and add their sums through LDS
// at the end, in a fixed order.
template <class V>
__device__ __forceinline__ V load_k(const char* row, int at, int k) {
  static_assert(sizeof(V) == 16, "");
  if (at + 16 <= k) return *reinterpret_cast<const V*>(row + at);
  V v = V{0, 0, 0, 0};
  if (at < k) {
    v = *reinterpret_cast<const V*>(row + at);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int b = k - at - 4 * w;
      if (b <= 0) v[w] = 0;
      else if (b < 4) v[w] &= (1u << (8 * b)) - 1;
    }
  }
  return v;
}

template <int FA, class C, bool TILE, int MT>
__global__ __launch_bounds__(256) void product_few_kernel(const Product p) {
  __shared__ __align__(16) f32x4 sums[4][MT][64];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT;
  const int brow = std::min(n0 + r, p.n - 1);
  const char* b = p.b + brow * p.ldb;
  const char* a[MT];
  int am[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    am[j] = std::min(m0 + 16 * j + r, p.m - 1);
    a[j] = p.a + am[j] * p.lda;
  }
  f32x4 acc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) acc[j] = f32x4{0, 0, 0, 0};
  const int steps = (p.k + kStepBytes - 1) / kStepBytes;
#pragma unroll 4
  for (int step = wave; step < steps; step += 4) {
    const int at = step * kStepBytes + g * 32;
    const i32x4 b0 = load_k<i32x4>(b, at, p.k), b1 = load_k<i32x4>(b, at + 16, p.k);
    const i32x8 bv = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
    float sn[4];
    if constexpr (TILE) {
      sn[0] = p.sb[static_cast<int64_t>(step) * p.nb + n0 / 128];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) sn[i] = p.sb[static_cast<int64_t>(step) * p.nb + std::min(n0 + 4 * g + i, p.n - 1)];
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const i32x4 a0 = load_k<i32x4>(a[j], at, p.k), a1 = load_k<i32x4>(a[j], at + 16, p.k);
      const i32x8 av = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
      const float s = p.sa[static_cast<int64_t>(step) * p.m + am[j]];
      const f32x4 part = mfma8<FA>(bv, av);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = __builtin_fmaf(part[i], s * sn[TILE ? 0 : i], acc[j][i]);
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) sums[wave][j][lane] = acc[j];
  __syncthreads();
  // lane l of wave w finishes m tile w (of MT)
  for (int j = wave; j < MT; j += 4) {
    const f32x4 t = (sums[0][j][lane] + sums[1][j][lane]) + (sums[2][j][lane] + sums[3][j][lane]);
    const int m = m0 + 16 * j + r;
    if (m >= p.m) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + 4 * g + i;
      if (n >= p.n) continue;
      p.c[m * p.ldc + n] = static_cast<uint16_t>(bits_of(C{}, t[i]));
    }
  }
}

template <int FA, class C, bool TILE>
hipError_t launch(Product p, hipStream_t stream) {
  if (p.m <= 64) {
    const dim3 grid((p.n + 15) / 16, 1);
    if (p.m <= 16) product_few_kernel<FA, C, TILE, 1><<<grid, 256, 0, stream>>>(p);
    else if (p.m <= 32) product_few_kernel<FA, C, TILE, 2><<<grid, 256, 0, stream>>>(p);
    else product_few_kernel<FA, C, TILE, 4><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError();
  }
  auto tiles = [&](int bm, int bn) {
    p.tiles_m = (p.m + bm - 1) / bm;
    p.tiles_n = (p.n + bn - 1) / bn;
    p.band = std::min(8, p.tiles_m);
    return static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  };
  if (tiles(256, 256) >= 200) {
    product_kernel<FA, C, TILE, 256, 256, 2, 4><<<p.tiles_m * p.tiles_n, 512, 0, stream>>>(p);
  } else {
    const int64_t t = tiles(128, 128);
    product_kernel<FA, C, TILE, 128, 128, 2, 2><<<static_cast<unsigned>(t), 256, 0, stream>>>(p);
  }
  return hipGetLastError();
}

template <int FA, class C>
hipError_t launch_block(const Product& p, int block, hipStream_t stream) {
  return block == OPT8_FP8_BLOCK_TILE ? launch<FA, C, true>(p, stream) : launch<FA, C, false>(p, stream);
}

template <int FA>
hipError_t launch_type(const Product& p, int type, int block, hipStream_t stream) {
  if (type == OPT8_TYPE_BF16) return launch_block<FA, Bf16>(p, block, stream);
  return launch_block<FA, Fp16>(p, block, stream);
}

}  // namespace

hipError_t launch_fp8_matmul(const opt8_fp8_product& q, hipStream_t stream) {
  Product p;
  p.a = static_cast<const char*>(q.a);
  p.sa = q.scale_a;
  p.b = static_cast<const char*>(q.b);
  p.sb = q.scale_b;
  p.c = static_cast<uint16_t*>(q.c);
  p.lda = q.lda;
  p.ldb = q.ldb;
  p.ldc = q.ldc;
  p.m = static_cast<int>(q.m);
  p.n = static_cast<int>(q.n);
  p.k = static_cast<int>(q.k);
  p.nb = q.block_b == OPT8_FP8_BLOCK_TILE ? (p.n + 127) / 128 : p.n;
  p.tiles_m = p.tiles_n = p.band = 0;
  p.vec = reinterpret_cast<uintptr_t>(q.c) % 16 == 0 && q.ldc % 8 == 0;
  if (q.a_type == OPT8_TYPE_E5M2) return launch_type<1>(p, q.c_type, q.block_b, stream);
  return launch_type<0>(p, q.c_type, q.block_b, stream);
}

}  // namespace opt8
