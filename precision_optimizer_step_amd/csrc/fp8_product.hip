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
#include <type_traits>

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
  static_assert((BM + BN) / 64 == NW, "a wave loads 64 scales a step");
  constexpr int kTile = (BM + BN) * kStepBytes;
  constexpr int kCopy = kTile + (BM + BN) * 4;
  __shared__ __align__(16) char lds[2][kCopy];

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
  const int srow = scales_a ? m0 + wave * 64 + lane : n0 + (wave - BM / 64) * 64 + lane;
  const int64_t sstep = scales_a ? p.m : p.nb;
  const char* sbase = reinterpret_cast<const char*>(scales_a ? p.sa : p.sb);
  uint32_t soff = static_cast<uint32_t>((scales_a || !TILE) ? srow : srow / 128) * 4;
  if (srow >= (scales_a ? p.m : p.n)) soff = kOutOfRange;
  __amdgpu_buffer_rsrc_t srange;

  auto at_step = [&](int step) {
    la.at_step(step, p.k - step * kStepBytes);
    lb.at_step(step, p.k - step * kStepBytes);
    srange = buffer(sbase + step * sstep * 4, step < steps ? sstep * 4 : 0);
  };
  // the wave's load l of the step: its parts of A, of B, its scales
  constexpr int kA = BM / 8 / NW, kB = BN / 8 / NW, kAll = kA + kB + 1;
  const uint32_t copies = lds_address(lds);
  auto issue = [&](uint32_t to, int l) {
    if (l < kA) la.issue(to, l);
    else if (l < kA + kB) lb.issue(to + BM * kStepBytes, l - kA);
    else load_lds_4(srange, soff, to + kTile + wave * 256);
  };
  auto clear = [&](int step) {
    if (step + 1 == steps && (p.k & 15)) {
      char* t = lds[step & 1];
      clear_part_chunk<BM, 64 * NW>(t, p.k - step * kStepBytes);
      clear_part_chunk<BN, 64 * NW>(t + BM * kStepBytes, p.k - step * kStepBytes);
      __syncthreads();
    }
  };

  Reader<kRows, BM, MT / 2> ra;
  Reader<kRows, BN, 2> rb;
  ra.init(wm * (BM / WM));
  rb.init(wn * 64);
  const int mlane = 8 * ((lane & 15) >> 2) + (lane & 3);
  const float* lds_scales = reinterpret_cast<const float*>(lds[0] + kTile);
  constexpr int kCopyFloats = kCopy / 4;
  auto both = [](i32x4 lo, i32x4 hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); };
  f32x4 acc[MT][4];
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[j][q] = f32x4{0, 0, 0, 0};

  // Row j's fragment of A is in a[0] (j even), a[1] (odd) or a[2] (the last).
  // Before the last two rows everything of this copy has been read: there the
  // waves meet, the next copy is complete, this one is filled again, and the
  // next step's B and first row are read.  B alternates between two sets of
  // registers, so steps go in pairs (a step past the last one adds zeros).
  i32x8 a[3], b[2][4];
  float sa[3];
  auto slot = [](int j) { return j == MT - 1 ? 2 : j & 1; };
  auto read_a = [&](int step, int j) {
    const char* t = lds[0] + (step & 1) * kCopy;
    a[slot(j)] = both(ra.read(t, j, 0), ra.read(t, j, 1));
    sa[slot(j)] = lds_scales[(step & 1) * kCopyFloats + wm * (BM / WM) + (j >> 1) * 32 + 4 * (j & 1) + mlane];
  };
  auto read_b = [&](int step, int set, int q) {
    const char* t = lds[0] + (step & 1) * kCopy + BM * kStepBytes;
    b[set][q] = both(rb.read(t, q, 0), rb.read(t, q, 1));
  };
  auto run = [&](int step, auto set) {
    constexpr int S = decltype(set)::value;
    const float* sb = lds_scales + (step & 1) * kCopyFloats + BM + wn * 64;
    f32x4 sn[TILE ? 1 : 4];
    if constexpr (TILE) {
      sn[0][0] = sb[0];
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sn[q] = *reinterpret_cast<const f32x4*>(sb + (q >> 1) * 32 + 8 * (lane >> 4) + 4 * (q & 1));
    }
    // A part is added two matrix instructions after its own: next to it the
    // hardware's wait for its result (about 10 instructions) would be spent idle.
    f32x4 part[3];
    float s[2] = {0.0f, 0.0f};
    auto add = [&](int k) {
      const int j = k / 4, q = k % 4;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[j][q][i] = __builtin_fmaf(part[k % 3][i], TILE ? s[j & 1] : s[j & 1] * sn[TILE ? 0 : q][i], acc[j][q][i]);
      asm volatile("" : "+v"(acc[j][q]));   // here and not later: 64 parts would not fit the registers
    };
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      if (j == MT - 2) {
        wait_and_meet();
        clear(step + 1);
        at_step(step + 2);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (j < MT - 2) {
          if (q == 0) read_a(step, j + 1);
          if (q == 2 && j == MT - 3) read_a(step, MT - 1);
        } else {
          // the last two rows: 8 places for the loads, B and the next first row
          const int at = (j - (MT - 2)) * 4 + q;
#pragma unroll
          for (int l = 0; l < kAll; ++l)
            if (l * 6 / kAll == at) issue(copies + (step & 1) * kCopy, l);
          if (at >= 2 && at < 6) read_b(step + 1, 1 - S, at - 2);
          if (at == 6) read_a(step + 1, 0);
        }
        const int k = 4 * j + q;
        part[k % 3] = mfma8<FA>(b[S][q], a[slot(j)]);
        if (k >= 2) add(k - 2);
        if (q == 1) s[j & 1] = TILE ? sa[slot(j)] * sn[0][0] : sa[slot(j)];
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    add(4 * MT - 2);
    add(4 * MT - 1);
  };

  if (steps > 0) {
    at_step(0);
#pragma unroll
    for (int l = 0; l < kAll; ++l) issue(copies, l);
    at_step(1);
#pragma unroll
    for (int l = 0; l < kAll; ++l) issue(copies + kCopy, l);
    wait_and_meet<kAll>();
    clear(0);
#pragma unroll
    for (int q = 0; q < 4; ++q) read_b(0, 0, q);
    read_a(0, 0);
    for (int step = 0; step < steps; step += 2) {
      run(step, std::integral_constant<int, 0>{});
      run(step + 1, std::integral_constant<int, 1>{});
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load outlives the workgroup's LDS
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
        v[i] = acc[j][2 * q][i];
        v[4 + i] = acc[j][2 * q + 1][i];
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
