// Gated feed-forward block: h = act(x Wg^T) * (x Wu^T), and its backward pass.
#include <algorithm>
#include <type_traits>

#include "products_internal.h"
#include "tile_product.h"

namespace opt8 {
namespace {

using namespace tile;

// ------------------------------------------------------------- activations
// exp by the hardware's base-2 exponential of x*log2(e): about 2^-22 relative,
// far below a 16-bit result's half step.  sigmoid(-inf) = 0 and sigmoid(inf) = 1.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_fast(-x)); }

constexpr float kTanhA = 0.7978845608028654f;    // sqrt(2/pi)
constexpr float kTanhB = 0.044715f;

// Value and slope of the activation.  tanh form: (1 + tanh y)/2 = sigmoid(2y).
__device__ __forceinline__ void activate(float g, int act, float& value, float& slope) {
  if (act == OPT8_ACT_SILU) {
    const float p = sigmoid(g);
    value = g * p;
    slope = p * __builtin_fmaf(g, 1.0f - p, 1.0f);
  } else if (act == OPT8_ACT_GELU) {
    const float below = 0.5f * erfcf(-0.70710678118654752f * g);
    value = g * below;
    slope = __builtin_fmaf(g * 0.39894228040143268f, exp_fast(-0.5f * g * g), below);
  } else {
    const float y = kTanhA * g * __builtin_fmaf(kTanhB * g, g, 1.0f);
    const float p = sigmoid(2.0f * y);
    value = g * p;
    slope = __builtin_fmaf(2.0f * g * p * (1.0f - p), kTanhA * __builtin_fmaf(3.0f * kTanhB * g, g, 1.0f), p);
  }
}
__device__ __forceinline__ float activate(float g, int act) {
  float value, slope;
  activate(g, act, value, slope);
  return value;
}

// ------------------------------------------------------------- tiled products
// The steps of one tile: both operands' loads are queued by issue(step), A lies
// first in a copy.  acc[q][j]: matrix tile q of the wave's two 32-column groups
// (n side), matrix tile j of its rows.
template <class T, Layout LA, Layout LB, int BM, int BN, int WM, class Issue, class Last>
__device__ __forceinline__ void multiply(char (*lds)[(BM + BN) * kStepBytes], int first, int steps,
                                         int mrow, int ncol0, int ncol1, Issue&& issue, Last&& last,
                                         f32x4 (&acc)[4][BM / WM / 16]) {
  constexpr int MT = BM / WM / 16;
  Reader<LA, BM, MT / 2> ra;
  Reader<LB, BN, 1> rb0, rb1;
  ra.init(mrow);
  rb0.init(ncol0);
  rb1.init(ncol1);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  if (steps > 0) issue(first, lds[0]);
  for (int s = 0; s < steps; ++s) {
    wait_and_meet();
    if (s + 1 < steps) issue(first + s + 1, lds[(s + 1) & 1]);
    char* t = lds[s & 1];
    if (s + 1 == steps) last(t);
    const char* tb = t + BM * kStepBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x4 b[4] = {rb0.read(tb, 0, h), rb0.read(tb, 1, h), rb1.read(tb, 0, h), rb1.read(tb, 1, h)};
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const i32x4 a = ra.read(t, j, h);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q][j] = mfma16<T>(b[q], a, acc[q][j]);
      }
    }
  }
}

// m (within the workgroup's tile) of matrix tile j, for this lane.
__device__ __forceinline__ int row_of(int mrow, int j) {
  const int lane = threadIdx.x & 63;
  return mrow + (j >> 1) * 32 + 4 * (j & 1) + 8 * ((lane & 15) >> 2) + (lane & 3);
}
template <int MT>
__device__ __forceinline__ void take8(const f32x4 (&acc)[4][MT], int group, int j, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = acc[2 * group][j][i];
    v[4 + i] = acc[2 * group + 1][j][i];
  }
}

struct Forward {
  const char* x;
  const char* wg;
  const char* wu;
  uint16_t* h;
  uint16_t* gate;
  uint16_t* up;
  int64_t ldx, ldw;     // bytes
  int64_t ldh, ldg;     // elements
  int rows, d, f, act;
  int tiles_m, tiles_n, band;
  bool vec;
};

// A BM x BN tile of B holds BN/2 rows of Wg and the same rows of Wu; a wave
// takes 32 of each, so g and u of one h meet in one lane.
template <class T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void gated_forward_kernel(const Forward p) {
  constexpr int NW = WM * WN, MT = BM / WM / 16, HALF = BN / 2;
  static_assert(BN / WN == 64 && NW % 2 == 0, "");
  __shared__ __align__(16) char lds[2][(BM + BN) * kStepBytes];
  int tm, tn;
  tile_of_group(p.tiles_m, p.tiles_n, p.band, tm, tn);
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int mrow = (wave / WN) * (BM / WM), wn = wave % WN;
  const int m0 = tm * BM, f0 = tn * HALF;
  const int64_t kbytes = 2 * int64_t{p.d}, kround = (kbytes + 15) & ~int64_t{15};
  Loader<kRows, BM, NW> la;
  Loader<kRows, HALF, NW / 2> lb;
  la.init(p.x + m0 * p.ldx, p.ldx, (std::min(BM, p.rows - m0) - 1) * p.ldx + kround, 0, wave);
  const bool second = wave >= NW / 2;
  lb.init((second ? p.wu : p.wg) + f0 * p.ldw, p.ldw, (std::min(HALF, p.f - f0) - 1) * p.ldw + kround, 0,
          second ? wave - NW / 2 : wave);
  const int bto = (BM + (second ? HALF : 0)) * kStepBytes;
  auto issue = [&](int step, char* to) {
    la.issue(to, step, kbytes);
    lb.issue(to + bto, step, kbytes);
  };
  const int steps = static_cast<int>((kbytes + kStepBytes - 1) / kStepBytes);
  auto last = [&](char* t) {
    if (kbytes & 15) {
      clear_part_chunk<BM + BN, 64 * NW>(t, static_cast<int>(kbytes - (steps - 1) * kStepBytes));
      __syncthreads();
    }
  };
  f32x4 acc[4][MT];
  multiply<T, kRows, kRows, BM, BN, WM>(lds, 0, steps, mrow, wn * 32, HALF + wn * 32, issue, last, acc);

  const int n = f0 + wn * 32 + 8 * (lane >> 4);
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t m = m0 + row_of(mrow, j);
    if (m >= p.rows) continue;
    float g[8], u[8], h[8];
    take8(acc, 0, j, g);
    take8(acc, 1, j, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = activate(g[i], p.act) * u[i];
    store8<T>(p.h + m * p.ldh + n, h, p.f - n, p.vec);
    if (p.gate) {
      store8<T>(p.gate + m * p.ldg + n, g, p.f - n, p.vec);
      store8<T>(p.up + m * p.ldg + n, u, p.f - n, p.vec);
    }
  }
}

// Few rows: the time is that of reading both weights.  A workgroup owns 16
// columns of h; its 4 waves take every fourth 64 of k straight from memory and
// add their sums through LDS in a fixed order.
__device__ __forceinline__ i32x4 load_part(const char* row, int64_t at, int64_t bytes) {
  if (at + 16 <= bytes) return *reinterpret_cast<const i32x4*>(row + at);
  i32x4 v = i32x4{0, 0, 0, 0};
  if (at < bytes) {
    v = *reinterpret_cast<const i32x4*>(row + at);
    const int n = static_cast<int>(bytes - at);   // even
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (n - 4 * w <= 0) v[w] = 0;
      else if (n - 4 * w < 4) v[w] &= 0xffff;
    }
  }
  return v;
}

template <class T, int MT>
__global__ __launch_bounds__(256) void gated_forward_few_kernel(const Forward p) {
  __shared__ __align__(16) f32x4 sums[4][2][MT][64];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int64_t row = std::min(n0 + r, p.f - 1), bytes = 2 * int64_t{p.d};
  const char* wg = p.wg + row * p.ldw;
  const char* wu = p.wu + row * p.ldw;
  const char* x[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) x[j] = p.x + std::min(16 * j + r, p.rows - 1) * p.ldx;
  f32x4 acc[2][MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) acc[0][j] = acc[1][j] = f32x4{0, 0, 0, 0};
  const int steps = static_cast<int>((bytes + kStepBytes - 1) / kStepBytes);
#pragma unroll 4
  for (int step = wave; step < steps; step += 4) {
    const int64_t at = int64_t{step} * kStepBytes + g * 32;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const i32x4 bg = load_part(wg, at + 16 * h, bytes), bu = load_part(wu, at + 16 * h, bytes);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const i32x4 a = load_part(x[j], at + 16 * h, bytes);
        acc[0][j] = mfma16<T>(bg, a, acc[0][j]);
        acc[1][j] = mfma16<T>(bu, a, acc[1][j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    sums[wave][0][j][lane] = acc[0][j];
    sums[wave][1][j][lane] = acc[1][j];
  }
  __syncthreads();
  for (int j = wave; j < MT; j += 4) {
    f32x4 t[2];
#pragma unroll
    for (int w = 0; w < 2; ++w)
      t[w] = (sums[0][w][j][lane] + sums[1][w][j][lane]) + (sums[2][w][j][lane] + sums[3][w][j][lane]);
    const int64_t m = 16 * j + r;
    if (m >= p.rows) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + 4 * g + i;
      if (n >= p.f) continue;
      p.h[m * p.ldh + n] = static_cast<uint16_t>(bits_of(T{}, activate(t[0][i], p.act) * t[1][i]));
      if (p.gate) {
        p.gate[m * p.ldg + n] = static_cast<uint16_t>(bits_of(T{}, t[0][i]));
        p.up[m * p.ldg + n] = static_cast<uint16_t>(bits_of(T{}, t[1][i]));
      }
    }
  }
}

// ------------------------------------------------------------- backward
struct Backward {
  const uint16_t* dh;
  const char* x;
  const char* wg;
  const char* wu;
  const uint16_t* gate;
  const uint16_t* up;
  uint16_t* dx;
  uint16_t* dwg;
  uint16_t* dwu;
  char* both;           // [rows][2*width]: dg, then du
  int64_t rows, width;  // width: f rounded up to 64
  int64_t ldx, ldw;     // bytes
  int64_t lddh, ldg, lddx, lddw;
  int d, f, act;
  int tiles_m, tiles_n, band;
  bool vec;
};

// dg and du, rounded to the type that the products take, zeros in the columns
// from f to width; 8 columns a thread.
template <class T>
__global__ __launch_bounds__(256) void gated_slopes_kernel(const Backward p) {
  const int64_t per = p.width / 8;
  const int64_t total = p.rows * per;
  for (int64_t at = int64_t{blockIdx.x} * 256 + threadIdx.x; at < total; at += int64_t{gridDim.x} * 256) {
    const int64_t m = at / per, n = (at - m * per) * 8;
    float dg[8], du[8];
    const uint16_t* a = p.dh + m * p.lddh + n;
    const uint16_t* b = p.gate + m * p.ldg + n;
    const uint16_t* c = p.up + m * p.ldg + n;
    i16x8 ra = {}, rb = {}, rc = {};
    if (n + 8 <= p.f) {
      ra = *reinterpret_cast<const i16x8*>(a);
      rb = *reinterpret_cast<const i16x8*>(b);
      rc = *reinterpret_cast<const i16x8*>(c);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n + i < p.f) {
          ra[i] = a[i];
          rb[i] = b[i];
          rc[i] = c[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float dh = value_of<T>(static_cast<uint16_t>(ra[i]));
      float value, slope;
      activate(value_of<T>(static_cast<uint16_t>(rb[i])), p.act, value, slope);
      dg[i] = dh * value_of<T>(static_cast<uint16_t>(rc[i])) * slope;
      du[i] = dh * value;
    }
    uint16_t* o = reinterpret_cast<uint16_t*>(p.both) + m * 2 * p.width + n;
    store8<T>(o, dg, 8, true);
    store8<T>(o + p.width, du, 8, true);
  }
}

// (The bodies of the next two are for the device pass alone: the host pass of
// this compiler leaves out the stubs of some of their instances otherwise.)
//
// dx = [dg du] [Wg; Wu]: k runs along the rows of the weights.
template <class T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void gated_dx_kernel(const Backward p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = WM * WN, MT = BM / WM / 16;
  static_assert(BN / WN == 64, "");
  __shared__ __align__(16) char lds[2][(BM + BN) * kStepBytes];
  int tm, tn;
  tile_of_group(p.tiles_m, p.tiles_n, p.band, tm, tn);
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int mrow = (wave / WN) * (BM / WM), wn = wave % WN;
  const int64_t m0 = int64_t{tm} * BM;
  const int n0 = tn * BN;
  const int64_t lda = 4 * p.width, kbytes = lda;
  Loader<kRows, BM, NW> la;
  Loader<kCols, BN, NW> lg, lu;
  la.init(p.both + m0 * lda, lda, std::min<int64_t>(BM, p.rows - m0) * lda, 0, wave);
  const int64_t climit = (p.f - 1) * p.ldw + ((2 * int64_t{p.d} + 15) & ~int64_t{15}) - 2 * n0;
  lg.init(p.wg + 2 * n0, p.ldw, climit, p.d - n0, wave);
  lu.init(p.wu + 2 * n0, p.ldw, climit, p.d - n0, wave);
  const int half = static_cast<int>(p.width / 64);
  auto issue = [&](int step, char* to) {
    la.issue(to, step, kbytes);
    if (step < half) lg.issue(to + BM * kStepBytes, step, 0);
    else lu.issue(to + BM * kStepBytes, step - half, 0);
  };
  f32x4 acc[4][MT];
  multiply<T, kRows, kCols, BM, BN, WM>(lds, 0, 2 * half, mrow, wn * 64, wn * 64 + 32, issue, [](char*) {}, acc);
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t m = m0 + row_of(mrow, j);
    if (m >= p.rows) continue;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int n = n0 + wn * 64 + 32 * q + 8 * (lane >> 4);
      float v[8];
      take8(acc, q, j, v);
      store8<T>(p.dx + m * p.lddx + n, v, p.d - n, p.vec);
    }
  }
#endif
}

// dWg = dg^T x and dWu = du^T x: k is the rows (tokens) of both operands.
template <class T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void gated_dw_kernel(const Backward p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = WM * WN, MT = BM / WM / 16;
  static_assert(BN / WN == 64, "");
  __shared__ __align__(16) char lds[2][(BM + BN) * kStepBytes];
  int tm, tn;
  tile_of_group(p.tiles_m, p.tiles_n, p.band, tm, tn);
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int mrow = (wave / WN) * (BM / WM), wn = wave % WN;
  const int one = p.tiles_m / 2;
  const bool second = tm >= one;
  const int f0 = (second ? tm - one : tm) * BM, n0 = tn * BN;
  const int64_t lda = 4 * p.width;
  Loader<kCols, BM, NW> la;
  Loader<kCols, BN, NW> lb;
  const int64_t off = 2 * (f0 + (second ? p.width : 0));
  la.init(p.both + off, lda, p.rows * lda - off, p.width - f0, wave);
  lb.init(p.x + 2 * n0, p.ldx, (p.rows - 1) * p.ldx + ((2 * int64_t{p.d} + 15) & ~int64_t{15}) - 2 * n0, p.d - n0, wave);
  auto issue = [&](int step, char* to) {
    la.issue(to, step, 0);
    lb.issue(to + BM * kStepBytes, step, 0);
  };
  const int steps = static_cast<int>((p.rows + 63) / 64);
  f32x4 acc[4][MT];
  multiply<T, kCols, kCols, BM, BN, WM>(lds, 0, steps, mrow, wn * 64, wn * 64 + 32, issue, [](char*) {}, acc);
  uint16_t* out = second ? p.dwu : p.dwg;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t m = f0 + row_of(mrow, j);
    if (m >= p.f) continue;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int n = n0 + wn * 64 + 32 * q + 8 * (lane >> 4);
      float v[8];
      take8(acc, q, j, v);
      store8<T>(out + m * p.lddw + n, v, p.d - n, p.vec);
    }
  }
#endif
}

bool wide(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * 2 % 16 == 0; }

template <class T>
hipError_t forward(Forward p, hipStream_t stream) {
  if (p.rows <= 64) {
    const unsigned grid = static_cast<unsigned>((p.f + 15) / 16);
    if (p.rows <= 16) gated_forward_few_kernel<T, 1><<<grid, 256, 0, stream>>>(p);
    else if (p.rows <= 32) gated_forward_few_kernel<T, 2><<<grid, 256, 0, stream>>>(p);
    else gated_forward_few_kernel<T, 4><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError();
  }
  auto tiles = [&](int bm, int bn) {
    p.tiles_m = (p.rows + bm - 1) / bm;
    p.tiles_n = (p.f + bn / 2 - 1) / (bn / 2);
    p.band = std::min(8, p.tiles_m);
    return static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  };
  if (const int64_t t = tiles(256, 256); t >= 200)
    gated_forward_kernel<T, 256, 256, 2, 4><<<static_cast<unsigned>(t), 512, 0, stream>>>(p);
  else
    gated_forward_kernel<T, 128, 128, 2, 2><<<static_cast<unsigned>(tiles(128, 128)), 256, 0, stream>>>(p);
  return hipGetLastError();
}

template <class T>
hipError_t backward(Backward p, hipStream_t stream) {
  const int64_t chunks = p.rows * (p.width / 8);
  if (chunks > 0) {
    gated_slopes_kernel<T><<<static_cast<unsigned>(std::min<int64_t>((chunks + 255) / 256, 1 << 20)), 256, 0, stream>>>(p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  auto tiles = [&](int64_t m, int64_t n, int b) {
    p.tiles_m = static_cast<int>((m + b - 1) / b);
    p.tiles_n = static_cast<int>((n + b - 1) / b);
    return static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  };
  if (p.dx && p.rows > 0) {
    p.vec = wide(p.dx, p.lddx);
    if (tiles(p.rows, p.d, 256) >= 200) {
      p.band = std::min(8, p.tiles_m);
      gated_dx_kernel<T, 256, 256, 2, 4><<<p.tiles_m * p.tiles_n, 512, 0, stream>>>(p);
    } else {
      tiles(p.rows, p.d, 128);
      p.band = std::min(8, p.tiles_m);
      gated_dx_kernel<T, 128, 128, 2, 2><<<p.tiles_m * p.tiles_n, 256, 0, stream>>>(p);
    }
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (p.dwg) {
    p.vec = wide(p.dwg, p.lddw) && wide(p.dwu, p.lddw);
    if (2 * tiles(p.f, p.d, 256) >= 200) {
      p.tiles_m *= 2;
      p.band = std::min(8, p.tiles_m);
      gated_dw_kernel<T, 256, 256, 2, 4><<<p.tiles_m * p.tiles_n, 512, 0, stream>>>(p);
    } else {
      tiles(p.f, p.d, 128);
      p.tiles_m *= 2;
      p.band = std::min(8, p.tiles_m);
      gated_dw_kernel<T, 128, 128, 2, 2><<<p.tiles_m * p.tiles_n, 256, 0, stream>>>(p);
    }
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_gated_ffn_forward(const opt8_gated_ffn& a, hipStream_t stream) {
  Forward p;
  p.x = static_cast<const char*>(a.x);
  p.wg = static_cast<const char*>(a.w_gate);
  p.wu = static_cast<const char*>(a.w_up);
  p.h = static_cast<uint16_t*>(a.h);
  p.gate = static_cast<uint16_t*>(a.gate);
  p.up = static_cast<uint16_t*>(a.up);
  p.ldx = 2 * a.ldx;
  p.ldw = 2 * a.ldw;
  p.ldh = a.ldh;
  p.ldg = a.ldg;
  p.rows = static_cast<int>(a.rows);
  p.d = static_cast<int>(a.d);
  p.f = static_cast<int>(a.f);
  p.act = a.act;
  p.tiles_m = p.tiles_n = p.band = 0;
  p.vec = wide(a.h, a.ldh) && (!a.gate || (wide(a.gate, a.ldg) && wide(a.up, a.ldg)));
  return a.type == OPT8_TYPE_BF16 ? forward<Bf16>(p, stream) : forward<Fp16>(p, stream);
}

hipError_t launch_gated_ffn_backward(const opt8_gated_ffn_grad& a, hipStream_t stream) {
  Backward p;
  p.dh = static_cast<const uint16_t*>(a.dh);
  p.x = static_cast<const char*>(a.x);
  p.wg = static_cast<const char*>(a.w_gate);
  p.wu = static_cast<const char*>(a.w_up);
  p.gate = static_cast<const uint16_t*>(a.gate);
  p.up = static_cast<const uint16_t*>(a.up);
  p.dx = static_cast<uint16_t*>(a.dx);
  p.dwg = static_cast<uint16_t*>(a.dw_gate);
  p.dwu = static_cast<uint16_t*>(a.dw_up);
  p.both = static_cast<char*>(a.workspace);
  p.rows = a.rows;
  p.width = gated_width(a.f);
  p.ldx = 2 * a.ldx;
  p.ldw = 2 * a.ldw;
  p.lddh = a.lddh;
  p.ldg = a.ldg;
  p.lddx = a.lddx;
  p.lddw = a.lddw;
  p.d = static_cast<int>(a.d);
  p.f = static_cast<int>(a.f);
  p.act = a.act;
  p.tiles_m = p.tiles_n = p.band = 0;
  p.vec = false;
  return a.type == OPT8_TYPE_BF16 ? backward<Bf16>(p, stream) : backward<Fp16>(p, stream);
}

}  // namespace opt8
