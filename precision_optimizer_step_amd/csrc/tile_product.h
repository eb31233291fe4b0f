// Tiled matrix products on the gfx950 matrix cores: C[m][n] = sum_k A(m,k)*B(n,k),
// one workgroup per BM x BN tile of C.  Shared by the 8-bit block-scaled
// product (fp8_product.hip) and the gated feed-forward block (gated_ffn.hip).
//
// A step of the contraction is 128 bytes of k (64 16-bit or 128 8-bit values).
// Its two operand tiles lie in LDS twice: while the waves multiply one copy,
// direct global-to-LDS loads fill the other, so a tile's latency has a whole
// step to pass and no register holds it on the way.  One barrier a step.
//
// Operand tiles in LDS, both swizzled so that neither the loads' linear
// writes nor the fragment reads meet bank conflicts (16-byte chunks; the loads
// write LDS in lane order, so it is the lane's global address that is permuted):
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

enum Layout : int { kRows = 0, kCols = 1 };

constexpr int kStepBytes = 128;
constexpr uint32_t kOutOfRange = 0x80000000u;   // an offset past every buffer's range (at most 2^31 - 1 bytes)

__device__ __forceinline__ constexpr int key(int row) { return (row & 3) | ((row >> 1) & 4); }

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

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

  // first: the wave's first load among this operand's
  __device__ __forceinline__ void init(const char* b, int64_t ld_, int64_t limit_, int64_t cols_left, int wave) {
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
  }
  // loads of step `step` into the LDS tile at `to`; kbytes: length of the contraction in bytes (kRows)
  __device__ __forceinline__ void issue(char* to, int step, int64_t kbytes) const {
    if constexpr (L == kRows) {
      const auto r = buffer(base, limit);
      const int soff = step * kStepBytes;
      const bool whole = soff + kStepBytes <= kbytes;
      const int lane = threadIdx.x & 63;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        uint32_t v = voff[j];
        if (!whole) {
          const int at = lds0 + j * 1024 + lane * 16;
          const int chunk = ((at >> 4) & 7) ^ key(at >> 7);
          if (soff + chunk * 16 >= kbytes) v = kOutOfRange;
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(to + lds0 + j * 1024), 16, v, soff, 0, 0);
      }
    } else {
      const int64_t skip = static_cast<int64_t>(step) * 64 * ld;
      const auto r = buffer(base + skip, limit - skip);
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(to + lds0 + j * 1024), 16, voff[j], 0, 0, 0);
    }
  }
};

// Clears the bytes of k at and past `kbytes` in the one 16-byte chunk of each
// row that holds both kinds (an operand whose k does not end on 16 bytes).
template <int ROWS, int THREADS>
__device__ __forceinline__ void clear_part_chunk(char* t, int kbytes_in_step) {
  const int chunk = kbytes_in_step >> 4, keep = kbytes_in_step & 15;
  for (int row = threadIdx.x; row < ROWS; row += THREADS) {
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
// 128 products of 8-bit values a result; both operands hold the same order of k.
// FA: the format of A, 0 e4m3, 1 e5m2; B is e4m3.
template <int FA>
__device__ __forceinline__ f32x4 mfma8(i32x8 b, i32x8 a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{0, 0, 0, 0}, 0, FA, 0, 0, 0, 0);
}

__device__ __forceinline__ void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
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

// Stores 8 consecutive results, each rounded once (to nearest, ties to even);
// `left` of them exist.  vec: the matrix lets 16 bytes be stored at once.
template <class T>
__device__ __forceinline__ void store8(uint16_t* p, const float* v, int64_t left, bool vec) {
  if (vec && left >= 8) {
    i32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = static_cast<int>(bits_of(T{}, v[2 * i]) | (bits_of(T{}, v[2 * i + 1]) << 16));
    *reinterpret_cast<i32x4*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = static_cast<uint16_t>(bits_of(T{}, v[i]));
  }
}

}  // namespace tile
}  // namespace opt8
