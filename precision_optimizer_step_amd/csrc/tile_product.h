// Tiled matrix products on the gfx950 matrix cores: C[m][n] = sum_k A(m,k)*B(n,k),
// one workgroup per BM x BN tile of C.  Shared by the 8-bit block-scaled
// product (fp8_product.hip) and the gated feed-forward block (gated_ffn.hip).
//
// A step of the contraction is 128 bytes of k (64 16-bit or 128 8-bit values).
// Its two operand tiles lie in LDS twice: while the waves multiply one copy,
// direct global-to-LDS loads fill the other, so a tile's latency has most of a
// step to pass and no register holds it on the way.
//
// Operand tiles in LDS, both swizzled against bank conflicts between the loads'
// linear writes and the fragment reads (16-byte chunks; the loads write LDS in
// lane order, so it is the lane's global address that is permuted).  Counted: none
// for rows; for the transposing reads 1 to 2 cycles an access in tiles of 128 and
// 256 columns, 4.3 in tiles of 64, whose rows of 8 chunks leave the swizzle one bit of
// the row's number, the one that already chooses the half of a 256-byte line of
// banks (twice the passes of the wider tiles, counting addresses):
//  - rows: [tile row][8 chunks of k], chunk c at slot c ^ key(row);
//  - cols (16-bit, an operand whose k runs along the rows of its matrix):
//    [64 k][tile columns], chunk c at slot c ^ (key(k) << 2), read with the
//    transposing LDS load (ds_read_b64_tr_b16: 4 k x 16 columns per 16 lanes).
//
// Fragments.  Within each 32 rows of a wave's part, row r of matrix tile t
// (r < 16, t < 2) is tile row 8*(r/4) + 4*t + r%4.  The matrix instruction
// returns to lane l column l%16 and rows 4*(l/16) + i; with B as its first
// operand and A as its second a lane so holds, for one m, the 8 consecutive n
// 8*(l/16) + 0..7 of a 32-column group: one 16-byte store of a 16-bit result.
//
// Ends: an element past the operands' k is read as zero (a buffer load out of
// range returns zero), a row past the last one too.
#pragma once

#include <cstdint>
#include <type_traits>
#include <utility>

#include <hip/hip_runtime.h>

namespace opt8 {
namespace tile {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) short i16x4;
typedef __attribute__((ext_vector_type(8))) short i16x8;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

struct Bf16 {};
struct Fp16 {};

// f(0), f(1), ... f(N - 1), each with its number as a constant.
template <class F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
  each_of(std::make_integer_sequence<int, N>{}, f);
}

enum Layout : int { kRows = 0, kCols = 1 };

constexpr int kStepBytes = 128;
constexpr uint32_t kOutOfRange = 0x80000000u;   // an offset past every buffer's range (at most 2^31 - 1 bytes)

__device__ __forceinline__ constexpr int key(int row) { return (row & 3) | ((row >> 1) & 4); }

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)p));
}

__device__ __forceinline__ auto buffer(const void* p, int64_t bytes) {
  const int n = static_cast<int>(bytes < 0 ? 0 : (bytes > 0x7fffffff ? 0x7fffffff : bytes));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, n, 0x00020000);
}

// XCD-aware order of the tiles.  Workgroups go to the 8 XCDs in turn; each XCD
// takes a contiguous run of tiles, walked in bands of `band` tile rows, so that
// the tiles in flight on one XCD share operand rows through its own L2.
__device__ __forceinline__ void tile_of_group(int tiles_m, int tiles_n, int band, int& tm, int& tn) {
  const int total = tiles_m * tiles_n;
  const int bid = blockIdx.x;
  const int xcd = bid & 7, q = total >> 3, r = total & 7;
  const int id = xcd * q + (xcd < r ? xcd : r) + (bid >> 3);
  const int per = band * tiles_n;
  const int b = id / per, in = id - b * per;
  const int h = (tiles_m - b * band) < band ? (tiles_m - b * band) : band;
  tm = b * band + in % h;
  tn = in / h;
}

// One wave load of 4 bytes a lane into LDS at `to`; as Loader::issue, in asm.
__device__ __forceinline__ void load_lds_4(__amdgpu_buffer_rsrc_t range, uint32_t off, uint32_t to) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(range));
#endif
}

// One operand's tile loads.  SIZE rows (or columns) of the tile, NW waves.
template <Layout L, int SIZE, int NW>
struct Loader {
  static constexpr int kLoads = SIZE / 8 / NW;      // 1 KiB wave loads each
  static_assert(SIZE % (8 * NW) == 0, "whole wave loads");
  static constexpr int kRowBytes = L == kRows ? kStepBytes : SIZE * 2;
  static constexpr int kChunks = kRowBytes / 16;
  const char* base;       // kRows: (row 0, k 0) of the tile; kCols: (k 0, column 0)
  int64_t ld;             // bytes between rows of the matrix
  int64_t limit;          // bytes from base to the end of the operand
  uint32_t voff[kLoads];
  int lds0;               // of this wave's first load
  __amdgpu_buffer_rsrc_t range;
  int soff;

  // cols_left (kCols): columns from the tile's first to the operand's last
  __device__ __forceinline__ void init(const char* b, int64_t ld_, int64_t limit_, int cols_left, int wave) {
    base = b;
    ld = ld_;
    limit = limit_;
    const int lane = threadIdx.x & 63;
    lds0 = wave * kLoads * 1024;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int at = (wave * kLoads + j) * 1024 + lane * 16;
      const int row = at / kRowBytes, slot = (at % kRowBytes) / 16;
      const int chunk = slot ^ (L == kRows ? key(row) : ((key(row) << 2) & (kChunks - 1)));
      voff[j] = static_cast<uint32_t>(row * ld) + chunk * 16;
      if (L == kCols && chunk * 8 >= cols_left) voff[j] = kOutOfRange;
    }
    range = buffer(base, limit);
    soff = 0;
  }
  // Makes `step` the one that issue() loads.  left (kRows): bytes of k from its
  // start; where they end inside the step (the last one), its lanes past them are
  // turned to zeros.
  __device__ __forceinline__ void at_step(int step, int left) {
    if constexpr (L == kRows) {
      soff = step * kStepBytes;
      if (left < kStepBytes) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const int at = lds0 + j * 1024 + (threadIdx.x & 63) * 16;
          if ((((at >> 4) & 7) ^ key(at >> 7)) * 16 >= left) voff[j] = kOutOfRange;
        }
      }
    } else {
      const int64_t skip = static_cast<int64_t>(step) * 64 * ld;
      range = buffer(base + skip, limit - skip);
    }
  }
  // Load j of the step into the tile at LDS address `to`.  It returns no register, so
  // nothing but the waits written in this file has to know of it: in asm, since
  // after the builtin the compiler waits for it before every transposing read of
  // the other copy (8192 x 4096 x 32768: 3.87 ms against 1.75).  (m0, which it writes, is a reserved
  // register: the compiler keeps nothing in it and no other instruction here reads it.)
  __device__ __forceinline__ void issue(uint32_t to, int j) const {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_add_i32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(to + lds0), "v"(voff[j]), "s"(range), "s"(soff), "s"(1024 * j) : "scc");
#endif
  }
};

// Clears the bytes of k at and past `kbytes` in the one 16-byte chunk of each
// row that holds both kinds (an operand whose k does not end on 16 bytes).
template <int ROWS, int THREADS>
__device__ __forceinline__ void clear_part_chunk(char* t, int kbytes_in_step, int thread) {
  const int chunk = kbytes_in_step >> 4, keep = kbytes_in_step & 15;
  for (int row = thread; row < ROWS; row += THREADS) {
    uint32_t* p = reinterpret_cast<uint32_t*>(t + row * kStepBytes + ((chunk ^ key(row)) << 4));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int b = keep - 4 * w;
      if (b <= 0) p[w] = 0;
      else if (b < 4) p[w] &= (1u << (8 * b)) - 1;
    }
  }
}

// Two transposing LDS loads: 4 k of the lane's column each.  (The host pass of
// the compiler drops a kernel that names this builtin, so it sees none.)
__device__ __forceinline__ i32x4 transposed_8(const char* p, const char* q) {
#if defined(__HIP_DEVICE_COMPILE__)
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)q);
  const i16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(i32x4, v);
#else
  (void)p;
  (void)q;
  return i32x4{0, 0, 0, 0};
#endif
}

// Fragment reads of one operand: GROUPS 32-row groups starting at tile row `row0`.
template <Layout L, int SIZE, int GROUPS>
struct Reader;

template <int SIZE, int GROUPS>
struct Reader<kRows, SIZE, GROUPS> {
  int at;   // chunk lane/16 of the lane's row; chunk lane/16 + 4 is at ^ 64
  __device__ __forceinline__ void init(int row0) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    at = (row0 + 8 * (r >> 2) + (r & 3)) * kStepBytes + ((g ^ (r & 7)) << 4);
  }
  // half h (64 bytes of k) of matrix tile 2*group + t
  __device__ __forceinline__ i32x4 read(const char* t, int tile, int h) const {
    const int off = (tile >> 1) * 32 * kStepBytes + (tile & 1) * 4 * kStepBytes;
    return *reinterpret_cast<const i32x4*>(t + (h ? (at ^ 64) : at) + off);
  }
};

template <int SIZE, int GROUPS>
struct Reader<kCols, SIZE, GROUPS> {
  static constexpr int kRowBytes = SIZE * 2;
  int at[GROUPS];
  __device__ __forceinline__ void init(int col0) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int j = i >> 2, p = i & 3;
    const int k = ((j | ((g & 1) << 2)) << 2) & (kRowBytes / 16 - 1);
#pragma unroll
    for (int q = 0; q < GROUPS; ++q)
      at[q] = (8 * g + j) * kRowBytes + (((col0 / 8 + 4 * q) ^ k) + p) * 16;
  }
  __device__ __forceinline__ i32x4 read(const char* t, int tile, int h) const {
    const char* p = t + at[tile >> 1] + (tile & 1) * 8 + h * 32 * kRowBytes;
    return transposed_8(p, p + 4 * kRowBytes);
  }
};

template <class T>
__device__ __forceinline__ f32x4 mfma16(i32x4 b, i32x4 a, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mfma16<Bf16>(i32x4 b, i32x4 a, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mfma16<Fp16>(i32x4 b, i32x4 a, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
}
// x += b a.  The empty asm keeps the sum in the accumulation half of the register
// file: left alone, the compiler moves sums between the halves inside the loop
// (210 moves beside 128 matrix instructions).
template <class T>
__device__ __forceinline__ void mfma_add(f32x4& x, const i32x4& b, const i32x4& a) {
  x = mfma16<T>(b, a, x);
  asm volatile("" : "+a"(x));
}
// Orders the sums behind a wait longer than any of these instructions runs (4
// passes of 4 cycles): after writing zeros to them, and before reading them.
template <int MT, int NT>
__device__ __forceinline__ void settle(f32x4 (&acc)[MT][NT]) {
  asm volatile("s_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int q = 0; q < NT; ++q) asm volatile("" : "+a"(acc[j][q]));
  asm volatile("s_nop 7" ::: "memory");
}

// 128 products of 8-bit values a result; both operands hold the same order of k.
// FA: the format of A, 0 e4m3, 1 e5m2; B is e4m3.
template <int FA>
__device__ __forceinline__ f32x4 mfma8(i32x8 b, i32x8 a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{0, 0, 0, 0}, 0, FA, 0, 0, 0, 0);
}

// Waits until at most LEFT of the wave's loads are under way and its LDS reads
// have come back, then for the other waves.
template <int LEFT = 0>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// A tiling of a 16-bit product: S x S tiles, in each team of waves WM of them
// along the rows and WN along the columns, KG teams that take the steps in turn
// (each with copies of its own) and add their sums at the end.
template <int S, int KG>
struct Tiling {
  static constexpr int kSize = S, kTeams = KG;
  static constexpr int WM = 2, WN = S == 64 ? 1 : 2, NW = WM * WN;   // 32 x 64, 64 x 64 or 128 x 128 to a wave
  static constexpr int MT = S / WM / 16, NT = S / WN / 16;
  static constexpr int kThreads = 64 * NW * KG, kMinWaves = S == 256 ? 1 : 2;
  static constexpr int kCopy = 2 * S * kStepBytes;
  typedef char Lds[KG][2][kCopy];
};

// The steps of one tile.  at_step(s) turns both operands' loaders to the team's
// step s, issue(j, to, i) queues the wave's j-th load of A (i = 0, first in a
// copy) or B, last(t) finishes the last step's copy before it is read (called by
// every team at the same step).  The wave's rows of A start at `mrow`, its
// columns at `ncol0` (first half of them) and `ncol1`.  acc[j][q]: matrix tile j
// of the wave's rows, q of its columns.
//
// Half a step (32 k) is in registers while the other half is on its way from
// LDS, so between two barriers a wave has a whole step of matrix instructions
// to issue.  The barrier lies in the middle of a step: before it the wave has
// read all of its copy, after it the next copy is complete and this one free.
// at_step() is called for two steps past the last one too; their loads are out
// of range and bring zeros without touching memory, which is cheaper than
// leaving them out (a second copy of the loop's body).
//
// 256 x 256 tiles, 8192 x 4096, k = 32768: 1.46-1.57 ms, 1.40-1.50 PFLOP/s, the matrix
// core busy 77% of the cycles at 1.8 GHz (the package's power limit).
template <class T, class G, Layout LA, Layout LB, class Step, class Issue, class Last>
__device__ __forceinline__ void multiply(char (*lds)[G::kCopy], int steps, int mrow, int ncol0, int ncol1, Step&& at_step,
                                         Issue&& issue, Last&& last, f32x4 (&acc)[G::MT][G::NT]) {
  constexpr int S = G::kSize, MT = G::MT, NT = G::NT, kLoads = S / 8 / G::NW;
  Reader<LA, S, MT / 2> ra;
  Reader<LB, S, NT / 4> rb[2];
  ra.init(mrow);
  rb[0].init(ncol0);
  rb[1].init(ncol1);
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int q = 0; q < NT; ++q) acc[j][q] = f32x4{0, 0, 0, 0};
  if (steps <= 0) return;
  const uint32_t copies = lds_address(lds);
  settle(acc);
  at_step(0);
#pragma unroll
  for (int l = 0; l < 2 * kLoads; ++l) issue(l / 2, copies, l % 2);
  at_step(1);
#pragma unroll
  for (int l = 0; l < 2 * kLoads; ++l) issue(l / 2, copies + G::kCopy, l % 2);
  wait_and_meet<2 * kLoads>();
  if (steps == 1) last(lds[0]);
  i32x4 a[2][MT], b[2][NT];
  // Read r of a half step's MT + NT: what its first row of matrix tiles needs comes first.
  auto read = [&](const char* from, int h, int r) {
    if (r == 0) a[h][0] = ra.read(from, 0, h);
    else if (r <= NT) b[h][r - 1] = rb[(r - 1) / (NT / 2)].read(from + S * kStepBytes, (r - 1) % (NT / 2), h);
    else a[h][r - NT] = ra.read(from, r - NT, h);
  };
#pragma unroll
  for (int r = 0; r < MT + NT; ++r) read(lds[0], 0, r);
  // The matrix instructions of half a step, with what is to be read and loaded
  // spread between them by prepare(place): each runs 16 cycles and a single wave
  // issues an instruction every 4, so at most three fit behind one.
  constexpr int kPlaces = MT * NT, kReads = MT + NT, kAll = kReads + 2 * kLoads;
  auto half = [&](int h, auto&& prepare) {
    each<kPlaces>([&](auto place) {
      constexpr int i = decltype(place)::value, j = i / NT, q = i % NT;
      mfma_add<T>(acc[j][q], b[h][q], a[h][j]);
      prepare(place);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  for (int s = 0; s < steps; ++s) {
    const char* t = lds[s & 1];
    const char* next = lds[(s + 1) & 1];
    const uint32_t to = copies + (s & 1) * G::kCopy;
    if constexpr (kPlaces >= 64) {
      // 256 x 256.  Four waves' loads at one for every 2 matrix instructions are
      // twice what the CU's cache path takes (64 bytes a cycle), and the wave that
      // waits to issue one cannot issue matrix instructions either.  So the waves
      // meet in the first half too, once the copy has been read, and the loads that
      // fill it again go behind every sixth instruction from there on.
      constexpr int kMeet = 36, kEvery = 6, kEarly = (kPlaces - kMeet + kEvery - 1) / kEvery;
      half(0, [&](auto place) {
        constexpr int i = decltype(place)::value;
        if constexpr (i % 2 == 0 && i / 2 < kReads) read(t, 1, i / 2);
        if constexpr (i == kMeet) {
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
          at_step(s + 2);
        }
        if constexpr (i >= kMeet && (i - kMeet) % kEvery == 0) issue((i - kMeet) / kEvery / 2, to, (i - kMeet) / kEvery % 2);
      });
      wait_and_meet<kEarly>();
      if (s + 2 == steps) last(lds[(s + 1) & 1]);
      half(1, [&](auto place) {
        constexpr int i = decltype(place)::value, l = kEarly + i / kEvery;
        if constexpr (i % kEvery == 0 && l < 2 * kLoads) issue(l / 2, to, l % 2);
        if constexpr (i % 4 == 2) read(next, 0, i / 4);
      });
      static_assert(kPlaces / 4 == kReads && (2 * kLoads - kEarly - 1) * kEvery < kPlaces, "all is read and loaded");
    } else {
      // smaller tiles: other waves of the SIMD fill the gaps
      auto in_place = [&](auto place, auto count, auto&& f) {
        constexpr int i = decltype(place)::value, n = decltype(count)::value;
        constexpr int begin = (i * n + kPlaces - 1) / kPlaces, end = ((i + 1) * n + kPlaces - 1) / kPlaces;
#pragma unroll
        for (int o = begin; o < end; ++o) f(o);
      };
      half(0, [&](auto place) {
        in_place(place, std::integral_constant<int, kReads>{}, [&](int o) { read(t, 1, o); });
      });
      wait_and_meet();
      if (s + 2 == steps) last(lds[(s + 1) & 1]);
      at_step(s + 2);
      half(1, [&](auto place) {
        in_place(place, std::integral_constant<int, kAll>{}, [&](int o) {
          if (o < 2 * kLoads) issue(o / 2, to, o % 2);     // the longest way first
          else read(next, 0, o - 2 * kLoads);
        });
      });
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load outlives the workgroup's LDS
  settle(acc);
}

// Adds the teams' sums, in the order of the teams; every team gets the result.
template <int KG, int NW, int MT, int NT, class L>
__device__ __forceinline__ void add_teams(L& lds, int team, int wave, f32x4 (&acc)[MT][NT]) {
  if constexpr (KG > 1) {
    static_assert(sizeof(L) >= KG * NW * MT * NT * 64 * sizeof(f32x4), "the copies hold the sums");
    f32x4* sums = reinterpret_cast<f32x4*>(lds);
    const int lane = threadIdx.x & 63;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT * NT; ++t) sums[((team * NW + wave) * MT * NT + t) * 64 + lane] = acc[t / NT][t % NT];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT * NT; ++t) {
      f32x4 v = sums[(wave * MT * NT + t) * 64 + lane];
#pragma unroll
      for (int g = 1; g < KG; ++g) v += sums[((g * NW + wave) * MT * NT + t) * 64 + lane];
      acc[t / NT][t % NT] = v;
    }
  }
}

// m (within the workgroup's tile) of matrix tile j, for this lane.
__device__ __forceinline__ int row_of(int mrow, int j) {
  const int lane = threadIdx.x & 63;
  return mrow + (j >> 1) * 32 + 4 * (j & 1) + 8 * ((lane & 15) >> 2) + (lane & 3);
}
// The lane's 8 consecutive columns of a 32-column group.
template <int MT, int NT>
__device__ __forceinline__ void take8(const f32x4 (&acc)[MT][NT], int group, int j, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = acc[j][2 * group][i];
    v[4 + i] = acc[j][2 * group + 1][i];
  }
}

// ------------------------------------------------------------- 16-bit results
__device__ __forceinline__ uint32_t bits_of(Bf16, float x) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
__device__ __forceinline__ uint32_t bits_of(Fp16, float x) {
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}
template <class T> __device__ __forceinline__ float value_of(uint16_t b);
template <> __device__ __forceinline__ float value_of<Bf16>(uint16_t b) { return static_cast<float>(__builtin_bit_cast(__bf16, b)); }
template <> __device__ __forceinline__ float value_of<Fp16>(uint16_t b) { return static_cast<float>(__builtin_bit_cast(_Float16, b)); }

// Loads and stores of 16 bytes at any alignment of their elements: the hardware
// splits those that cross a line (n = 10941 results a row: 139 us with an element
// to a lane).
typedef i32x4 __attribute__((aligned(2))) i32x4_at2;
typedef f32x4 __attribute__((aligned(4))) f32x4_at4;

// The first `left` (at most 8) of 8 results.
__device__ __forceinline__ void store_some(uint16_t* p, i32x4 w, int64_t left) {
  if (left >= 8) {
    *reinterpret_cast<i32x4_at2*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
}
// 8 results, each rounded once (to nearest, ties to even).
template <class T>
__device__ __forceinline__ i32x4 packed(const float* v) {
  i32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = static_cast<int>(bits_of(T{}, v[2 * i]) | (bits_of(T{}, v[2 * i + 1]) << 16));
  return w;
}

// 16 rows (matrix tile j of the wave's) of NG 32-column groups, through LDS, so
// that a store instruction writes whole rows of 64*NG bytes: straight from the
// fragments it would write 64 bytes of each of 16 rows, half cache lines (3 x 268
// MB in 205 us more than one of them alone; so in 110).  `left` columns exist from
// out on.  Only the wave itself reads what it wrote, and LDS keeps a wave's order.
template <int NG> constexpr int kRowScratch = 16 * NG * 64;
template <class T, int NG>
__device__ __forceinline__ void store_rows(char* scratch, uint16_t* out, int64_t ld, int64_t rows, int left, int64_t m0,
                                           int mrow, int j, const float (&v)[NG][8]) {
  constexpr int kChunks = 4 * NG;      // of 16 bytes in a row
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  auto place = [](int row, int chunk) { return (row * kChunks + (chunk ^ (row & (kChunks - 1)))) * 16; };
  auto row_at = [&](int row) { return m0 + mrow + (j >> 1) * 32 + 4 * (j & 1) + 8 * (row >> 2) + (row & 3); };
#pragma unroll
  for (int q = 0; q < NG; ++q) *reinterpret_cast<i32x4*>(scratch + place(r, 4 * q + g)) = packed<T>(v[q]);
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int n = 0; n < 16 * kChunks / 64; ++n) {
    const int row = (n * 64 + lane) / kChunks, chunk = (n * 64 + lane) % kChunks;
    const i32x4 w = *reinterpret_cast<const i32x4*>(scratch + place(row, chunk));
    const int64_t m = row_at(row);
    if (m < rows) store_some(out + m * ld + chunk * 8, w, left - chunk * 8);
  }
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void store_some(float* p, const float* v, int64_t left) {
  if (left >= 8) {
    *reinterpret_cast<f32x4_at4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4_at4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = v[i];
  }
}

}  // namespace tile
}  // namespace opt8
