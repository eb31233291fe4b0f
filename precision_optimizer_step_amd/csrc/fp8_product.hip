// C = A B^T on 8-bit floating point operands with a scale for each 128 values of
// k: C[m][n] = sum_b (sa[b][m] * sb[b][n]) * sum_{k in b} A[m][k] B[n][k].
//
// Precision.  The 8-bit matrix instruction aligns each 8 products to the largest
// one and drops what lies 2^-13 below its power of two (measured: a term 2^-14 of
// another among the same 8 consecutive k is lost whole, in another 8 kept);
// sums of the 8s are fp32.  Measured on sums that cancel, in norm: 1e-5 of a result on
// normal values, 3e-5 where one channel in a hundred is 20 times as large, 1 to 3% of
// bf16's rounding and 7 to 20% of fp16's; at most 2^-13 * 7^(1/2) = 3.3e-4.
//
// Range.  The scales' product is formed first: one multiplication for four matrix
// instructions with TILE scales, where scaling by either in turn would double the
// vector ALU's work.  So it has to be a normal fp32 number.
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
};

// (The body is for the device pass alone: the host pass of this compiler
// otherwise leaves out the launch stubs of some instances.)
//
// One BM x BN tile of C, WM x WN waves.  The scales of a step's block of k lie
// in LDS beside its operand tiles, one for each row of either (TILE scales are
// spread over their rows by the loads' addresses).
//
// Every block's partial sums pass the vector ALU (4 fused multiply-adds a matrix
// instruction with TILE scales, and 4 products more with ROW ones), which cannot
// use accumulation registers: hence 128 x 64 results to a wave and two waves a
// SIMD.  8192 x 16384 x 4096, TILE: 479 us, 2.29 PFLOP/s, matrix core 61% busy at
// 1.8 GHz, a third of the waves' cycles at the barrier.  (The 256 x 256 kernel with ROW
// scales spills 4 registers, read again in a ragged last step and behind the loop alone.)
//
// KG > 1: KG teams of WM x WN waves share the tile's steps in turn, each with its
// own copies, and add their sums through LDS at the end, in a fixed order: for
// results too small to give every CU a tile.
template <int FA, class C, bool TILE, int BM, int BN, int WM, int WN, int KG = 1>
__global__ __launch_bounds__(64 * WM * WN * KG, 2) void product_kernel(const Product p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = WM * WN;
  constexpr int MT = BM / WM / 16;
  static_assert(BN / WN == 64, "a wave takes 64 columns");
  static_assert((BM + BN) / 64 == NW, "a wave loads 64 scales a step");
  constexpr int kTile = (BM + BN) * kStepBytes;
  constexpr int kCopy = kTile + (BM + BN) * 4;
  __shared__ __align__(16) char lds_all[KG][2][kCopy];

  int tm, tn;
  tile_of_group(p.tiles_m, p.tiles_n, p.band, tm, tn);
  const int lane = threadIdx.x & 63;
  const int team = KG > 1 ? wave_id() / NW : 0, wave = KG > 1 ? wave_id() % NW : wave_id();
  char(*lds)[kCopy] = lds_all[team];
  const int wm = wave / WN, wn = wave % WN;
  const int m0 = tm * BM, n0 = tn * BN;
  const int64_t kbytes = p.k, kround = (kbytes + 15) & ~int64_t{15};

  Loader<kRows, BM, NW> la;
  Loader<kRows, BN, NW> lb;
  la.init(p.a + m0 * p.lda, p.lda, (std::min(BM, p.m - m0) - 1) * p.lda + kround, 0, wave);
  lb.init(p.b + n0 * p.ldb, p.ldb, (std::min(BN, p.n - n0) - 1) * p.ldb + kround, 0, wave);
  const int all_steps = (p.k + kStepBytes - 1) / kStepBytes;
  const int steps = (all_steps + KG - 1) / KG;     // of each team: step s is s*KG + team of the product

  // this wave's 64 scales: of A's rows (waves 0 .. BM/64 - 1) or of B's
  const bool scales_a = wave < BM / 64;
  const int srow = scales_a ? m0 + wave * 64 + lane : n0 + (wave - BM / 64) * 64 + lane;
  const int64_t sstep = scales_a ? p.m : p.nb;
  const char* sbase = reinterpret_cast<const char*>(scales_a ? p.sa : p.sb);
  uint32_t soff = static_cast<uint32_t>((scales_a || !TILE) ? srow : srow / 128) * 4;
  if (srow >= (scales_a ? p.m : p.n)) soff = kOutOfRange;
  __amdgpu_buffer_rsrc_t srange;

  auto at_step = [&](int s) {
    const int step = s * KG + team;
    la.at_step(step, p.k - step * kStepBytes);
    lb.at_step(step, p.k - step * kStepBytes);
    srange = buffer(sbase + step * sstep * 4, step < all_steps ? sstep * 4 : 0);
  };
  // the wave's load l of the step: its parts of A, of B, its scales
  constexpr int kA = BM / 8 / NW, kB = BN / 8 / NW, kAll = kA + kB + 1;
  // With one workgroup to a CU (256 x 256), the loads of a step are more than the
  // CU's cache path takes (64 bytes a cycle) in the two rows behind the barrier,
  // and waves that wait to issue one stand still: some go to the next row (ROW, whose
  // rows last longer, 2: 120 us against 127 with 4 in the weight gradient's case).
  constexpr int kLater = MT == 8 ? (TILE ? 4 : 2) : 0, kNow = kAll - kLater;
  const uint32_t copies = lds_address(lds);
  auto issue = [&](uint32_t to, int l) {
    if (l < kA) la.issue(to, l);
    else if (l < kA + kB) lb.issue(to + BM * kStepBytes, l - kA);
    else load_lds_4(srange, soff, to + kTile + wave * 256);
  };
  auto clear = [&](int step) {
    if (step + 1 == steps && (p.k & 15)) {
      if (KG == 1 || step * KG + team + 1 == all_steps)
        clear_part_chunk<BM + BN, 64 * NW>(lds[step & 1], p.k - (all_steps - 1) * kStepBytes, threadIdx.x - team * 64 * NW);
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
        constexpr bool two = MT == 2;     // both rows are read at the end of the step before
        if (j == 0 && q * kLater % 4 == 0 && kLater)      // what was left of the next step's loads
          issue(copies + ((step + 1) & 1) * kCopy, kNow + q * kLater / 4);
        if (!two && j < MT - 2) {
          if (q == 0) read_a(step, j + 1);
          if (q == 2 && j == MT - 3) read_a(step, MT - 1);
        } else {
          // the last two rows: 8 places for the loads, B and the next first row
          const int at = (j - (MT - 2)) * 4 + q;
#pragma unroll
          for (int l = 0; l < kNow; ++l)
            if (l * 6 / kNow == at) issue(copies + (step & 1) * kCopy, l);
          if (at >= 2 && at < 6) read_b(step + 1, 1 - S, at - 2);
          if (!two && at == 6) read_a(step + 1, 0);
        }
        const int k = 4 * j + q;
        part[k % 3] = mfma8<FA>(b[S][q], a[slot(j)]);
        if (k >= 2) add(k - 2);
        if (q == 1) s[j & 1] = TILE ? sa[slot(j)] * sn[0][0] : sa[slot(j)];
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (MT == 2) {
      read_a(step + 1, 0);
      read_a(step + 1, 1);
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
    for (int l = 0; l < kNow; ++l) issue(copies + kCopy, l);
    wait_and_meet<kNow>();
    clear(0);
#pragma unroll
    for (int q = 0; q < 4; ++q) read_b(0, 0, q);
    read_a(0, 0);
    if constexpr (MT == 2) read_a(0, 1);
    for (int step = 0; step < steps; step += 2) {
      run(step, std::integral_constant<int, 0>{});
      run(step + 1, std::integral_constant<int, 1>{});
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load outlives the workgroup's LDS
  }

  // each team finishes its share of the 32-column groups
  add_teams<KG, NW, MT, 4>(lds_all, team, wave, acc);
  __syncthreads();       // other waves may still read what the results are staged in
  constexpr int NG = KG == 1 ? 2 : 1;
  char* scratch = lds_all[0][0] + (team * NW + wave) * kRowScratch<NG>;
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int q = 0; q < 2; q += NG) {
      if (KG > 1 && (2 * j + q) % KG != team) continue;
      const int n = n0 + wn * 64 + q * 32;
      float v[NG][8];
#pragma unroll
      for (int i = 0; i < NG; ++i) take8(acc, q + i, j, v[i]);
      if (n < p.n) store_rows<C, NG>(scratch, p.c + n, p.ldc, p.m, p.n - n, m0, wm * (BM / WM), j, v);
    }
#endif
}

// At most 16 rows (single tokens): the time is that of reading B, so nothing goes
// through LDS.  A workgroup owns 16 n; each of its 4 waves takes a quarter of k,
// in one piece, holds B's and A's fragments in registers straight from memory (a
// lane 32 bytes of a row's 128, four blocks under way at once) and adds its sums
// to the others' through LDS at the end, in a fixed order.  One row, n = 4096, k
// = 16384: 12.5 us, 5.4 TB/s.  Waves that take blocks in turn instead read all
// rows at one place of k at a time; where rows lie a power of two apart that
// is one memory channel: 21 us.
__device__ __forceinline__ i32x4 load_part(const char* row, int at, int k) {
  i32x4 v = i32x4{0, 0, 0, 0};
  if (at < k) v = *reinterpret_cast<const i32x4*>(row + at);
  if (at + 16 > k) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int b = k - at - 4 * w;
      if (b <= 0) v[w] = 0;
      else if (b < 4) v[w] &= (1u << (8 * b)) - 1;
    }
  }
  return v;
}

template <int FA, class C, bool TILE>
__global__ __launch_bounds__(256) void product_few_kernel(const Product p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kDepth = 4, kScales = TILE ? 1 : 4;
  __shared__ __align__(16) f32x4 sums[4][64];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int am = std::min(r, p.m - 1);
  const char* b = p.b + std::min(n0 + r, p.n - 1) * p.ldb + g * 32;
  const char* a = p.a + am * p.lda + g * 32;
  int bn[kScales];
#pragma unroll
  for (int i = 0; i < kScales; ++i) bn[i] = TILE ? n0 / 128 : std::min(n0 + 4 * g + i, p.n - 1);
  f32x4 acc = f32x4{0, 0, 0, 0};

  struct Block {
    i32x8 b, a;
    float sa, sb[kScales];
  };
  auto scales = [&](Block& x, int step) {
#pragma unroll
    for (int i = 0; i < kScales; ++i) x.sb[i] = p.sb[static_cast<int64_t>(step) * p.nb + bn[i]];
    x.sa = p.sa[static_cast<int64_t>(step) * p.m + am];
  };
  auto both = [](i32x4 lo, i32x4 hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); };
  auto whole = [&](const char* row, int step) {
    const i32x4* v = reinterpret_cast<const i32x4*>(row + step * kStepBytes);
    return both(v[0], v[1]);
  };
  auto load = [&](Block& x, int step) {
    x.b = whole(b, step);
    x.a = whole(a, step);
    scales(x, step);
  };
  auto add = [&](const Block& x) {
    const f32x4 part = mfma8<FA>(x.b, x.a);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(part[i], x.sa * x.sb[TILE ? 0 : i], acc[i]);
  };
  const int steps = p.k / kStepBytes;      // whole blocks
  int step = steps * wave / 4;
  const int end = steps * (wave + 1) / 4;
  for (; step + kDepth <= end; step += kDepth) {
    Block x[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth; ++i) load(x[i], step + i);
#pragma unroll
    for (int i = 0; i < kDepth; ++i) add(x[i]);
  }
  for (; step < end; ++step) {
    Block x;
    load(x, step);
    add(x);
  }
  if (wave == 3 && p.k % kStepBytes) {
    const int left = p.k % kStepBytes - g * 32;
    Block x;
    auto part = [&](const char* row) {
      return both(load_part(row + steps * kStepBytes, 0, left), load_part(row + steps * kStepBytes, 16, left));
    };
    x.b = part(b);
    x.a = part(a);
    scales(x, steps);
    add(x);
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave == 0 && r < p.m) {
    const f32x4 t = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + 4 * g + i;
      if (n < p.n) p.c[r * p.ldc + n] = static_cast<uint16_t>(bits_of(C{}, t[i]));
    }
  }
#endif
}

template <int FA, class C, bool TILE>
hipError_t launch(Product& p, hipStream_t stream) {
  if (p.m <= kFewRows) return queue(product_few_kernel<FA, C, TILE>, (p.n + 15) / 16, 256, stream, p);
  const int choice = fp8_choice(p.m, p.n, p.k, TILE), size = tile_size(choice);
  p.tiles_m = (p.m + size - 1) / size;
  p.tiles_n = (p.n + size - 1) / size;
  p.band = std::min(8, p.tiles_m);
  const unsigned grid = static_cast<unsigned>(tiles_of(p.m, p.n, size));
  switch (choice) {
    case kTile256: return queue(product_kernel<FA, C, TILE, 256, 256, 2, 4>, grid, 512, stream, p);
    case kTile128: return queue(product_kernel<FA, C, TILE, 128, 128, 2, 2>, grid, 256, stream, p);
    case kTile128Teams2: return queue(product_kernel<FA, C, TILE, 128, 128, 2, 2, 2>, grid, 512, stream, p);
    case kTile64Teams2: return queue(product_kernel<FA, C, TILE, 64, 64, 2, 1, 2>, grid, 256, stream, p);
    default: return queue(product_kernel<FA, C, TILE, 64, 64, 2, 1, 4>, grid, 512, stream, p);
  }
}

template <int FA, class C>
hipError_t launch_block(Product& p, int block, hipStream_t stream) {
  return block == OPT8_FP8_BLOCK_TILE ? launch<FA, C, true>(p, stream) : launch<FA, C, false>(p, stream);
}

template <int FA>
hipError_t launch_type(Product& p, int type, int block, hipStream_t stream) {
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
  if (q.a_type == OPT8_TYPE_E5M2) return launch_type<1>(p, q.c_type, q.block_b, stream);
  return launch_type<0>(p, q.c_type, q.block_b, stream);
}

}  // namespace opt8
