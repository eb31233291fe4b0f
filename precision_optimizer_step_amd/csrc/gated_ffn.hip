// Gated feed-forward block: h = act(x Wg^T) * (x Wu^T), and its backward pass.
//
// The bodies of the tiled kernels are for the device pass alone: the host pass of
// this compiler otherwise leaves out the launch stubs of some of their instances.
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
template <int ACT>
__device__ __forceinline__ void activate(float g, float& value, float& slope) {
  if constexpr (ACT == OPT8_ACT_SILU) {
    const float p = sigmoid(g);
    value = g * p;
    slope = p * __builtin_fmaf(g, 1.0f - p, 1.0f);
  } else if constexpr (ACT == OPT8_ACT_GELU) {
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
template <int ACT>
__device__ __forceinline__ float activate(float g) {
  float value, slope;
  activate<ACT>(g, value, slope);
  return value;
}
// Calls f with the activation as a constant: the choice is made once, so that
// the chains of neighbouring values overlap.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == OPT8_ACT_SILU) f(std::integral_constant<int, OPT8_ACT_SILU>{});
  else if (act == OPT8_ACT_GELU) f(std::integral_constant<int, OPT8_ACT_GELU>{});
  else f(std::integral_constant<int, OPT8_ACT_GELU_TANH>{});
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

// A tile holds B/2 rows of Wg and the same rows of Wu beside B rows of x; a
// wave takes as many columns of one as of the other, so g and u of one h meet
// in one lane.
template <class T, int B>
__global__ __launch_bounds__(256, B == 256 ? 1 : 2) void gated_forward_kernel(const Forward p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int T16 = B / 32, HALF = B / 2;
  __shared__ __align__(16) char lds[2][2 * B * kStepBytes];
  int tm, tn;
  tile_of_group(p.tiles_m, p.tiles_n, p.band, tm, tn);
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int mrow = (wave >> 1) * HALF, ncol = (wave & 1) * (HALF / 2);
  const int m0 = tm * B, f0 = tn * HALF;
  const int64_t kbytes = 2 * int64_t{p.d}, kround = (kbytes + 15) & ~int64_t{15};
  Loader<kRows, B, 4> la;
  Loader<kRows, HALF, 2> lb;
  la.init(p.x + m0 * p.ldx, p.ldx, (std::min(B, p.rows - m0) - 1) * p.ldx + kround, 0, wave);
  const bool second = wave >= 2;
  lb.init((second ? p.wu : p.wg) + f0 * p.ldw, p.ldw, (std::min(HALF, p.f - f0) - 1) * p.ldw + kround, 0, wave & 1);
  const int bto = (B + (second ? HALF : 0)) * kStepBytes;
  auto at_step = [&](int step) {
    const int left = static_cast<int>(kbytes) - step * kStepBytes;
    la.at_step(step, left);
    lb.at_step(step, left);
  };
  auto issue = [&](int j, uint32_t to, int i) {
    if (i == 0) la.issue(to, j);
    else lb.issue(to + bto, j);
  };
  const int steps = static_cast<int>((kbytes + kStepBytes - 1) / kStepBytes);
  auto last = [&](char* t) {
    if (kbytes & 15) {
      clear_part_chunk<2 * B, 256>(t, static_cast<int>(kbytes - (steps - 1) * kStepBytes), threadIdx.x);
      __syncthreads();
    }
  };
  f32x4 acc[T16][T16];
  multiply<T, kRows, kRows, B, B, 2, 2>(lds, 0, steps, mrow, ncol, HALF + ncol, at_step, issue, last, acc);

  with_act(p.act, [&](auto act) {
#pragma unroll
    for (int j = 0; j < T16; ++j) {
      const int64_t m = m0 + row_of(mrow, j);
      if (m >= p.rows) continue;
#pragma unroll
      for (int q = 0; q < T16 / 4; ++q) {
        const int n = f0 + ncol + 32 * q + 8 * (lane >> 4);
        float g[8], u[8], h[8];
        take8(acc, q, j, g);
        take8(acc, q + T16 / 4, j, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = activate<decltype(act)::value>(g[i]) * u[i];
        store8<T>(p.h + m * p.ldh + n, h, p.f - n, p.vec);
        if (p.gate) {
          store8<T>(p.gate + m * p.ldg + n, g, p.f - n, p.vec);
          store8<T>(p.up + m * p.ldg + n, u, p.f - n, p.vec);
        }
      }
    }
  });
#endif
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
      float value = 0.0f;
      with_act(p.act, [&](auto act) { value = activate<decltype(act)::value>(t[0][i]); });
      p.h[m * p.ldh + n] = static_cast<uint16_t>(bits_of(T{}, value * t[1][i]));
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
    with_act(p.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float dh = value_of<T>(static_cast<uint16_t>(ra[i]));
        float value, slope;
        activate<decltype(act)::value>(value_of<T>(static_cast<uint16_t>(rb[i])), value, slope);
        dg[i] = dh * value_of<T>(static_cast<uint16_t>(rc[i])) * slope;
        du[i] = dh * value;
      }
    });
    uint16_t* o = reinterpret_cast<uint16_t*>(p.both) + m * 2 * p.width + n;
    store8<T>(o, dg, 8, true);
    store8<T>(o + p.width, du, 8, true);
  }
}

// dx = [dg du] [Wg; Wu]: k runs along the rows of the weights.
template <class T, int B>
__global__ __launch_bounds__(256, B == 256 ? 1 : 2) void gated_dx_kernel(const Backward p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int T16 = B / 32, HALF = B / 2;
  __shared__ __align__(16) char lds[2][2 * B * kStepBytes];
  int tm, tn;
  tile_of_group(p.tiles_m, p.tiles_n, p.band, tm, tn);
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int mrow = (wave >> 1) * HALF, ncol = (wave & 1) * HALF;
  const int64_t m0 = int64_t{tm} * B;
  const int n0 = tn * B;
  const int64_t lda = 4 * p.width;
  Loader<kRows, B, 4> la;
  Loader<kCols, B, 4> lb;
  la.init(p.both + m0 * lda, lda, std::min<int64_t>(B, p.rows - m0) * lda, 0, wave);
  lb.init(p.wg + 2 * n0, p.ldw, (p.f - 1) * p.ldw + ((2 * int64_t{p.d} + 15) & ~int64_t{15}) - 2 * n0, p.d - n0, wave);
  const int half = static_cast<int>(p.width / 64);
  auto at_step = [&](int step) {
    la.at_step(step, (2 * half - step) * kStepBytes);
    lb.base = (step < half ? p.wg : p.wu) + 2 * n0;
    lb.at_step(step < half ? step : step - half, 0);
  };
  auto issue = [&](int j, uint32_t to, int i) {
    if (i == 0) la.issue(to, j);
    else lb.issue(to + B * kStepBytes, j);
  };
  f32x4 acc[T16][T16];
  multiply<T, kRows, kCols, B, B, 2, 2>(lds, 0, 2 * half, mrow, ncol, ncol + HALF / 2, at_step, issue, [](char*) {}, acc);
#pragma unroll
  for (int j = 0; j < T16; ++j) {
    const int64_t m = m0 + row_of(mrow, j);
    if (m >= p.rows) continue;
#pragma unroll
    for (int q = 0; q < T16 / 2; ++q) {
      const int n = n0 + ncol + 32 * q + 8 * (lane >> 4);
      float v[8];
      take8(acc, q, j, v);
      store8<T>(p.dx + m * p.lddx + n, v, p.d - n, p.vec);
    }
  }
#endif
}

// dWg = dg^T x and dWu = du^T x: k is the rows (tokens) of both operands.
template <class T, int B>
__global__ __launch_bounds__(256, B == 256 ? 1 : 2) void gated_dw_kernel(const Backward p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int T16 = B / 32, HALF = B / 2;
  __shared__ __align__(16) char lds[2][2 * B * kStepBytes];
  int tm, tn;
  tile_of_group(p.tiles_m, p.tiles_n, p.band, tm, tn);
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int mrow = (wave >> 1) * HALF, ncol = (wave & 1) * HALF;
  const int one = p.tiles_m / 2;
  const bool second = tm >= one;
  const int f0 = (second ? tm - one : tm) * B, n0 = tn * B;
  const int64_t lda = 4 * p.width;
  Loader<kCols, B, 4> la, lb;
  const int64_t off = 2 * (f0 + (second ? p.width : 0));
  la.init(p.both + off, lda, p.rows * lda - off, static_cast<int>(p.width) - f0, wave);
  lb.init(p.x + 2 * n0, p.ldx, (p.rows - 1) * p.ldx + ((2 * int64_t{p.d} + 15) & ~int64_t{15}) - 2 * n0, p.d - n0, wave);
  auto at_step = [&](int step) {
    la.at_step(step, 0);
    lb.at_step(step, 0);
  };
  auto issue = [&](int j, uint32_t to, int i) {
    if (i == 0) la.issue(to, j);
    else lb.issue(to + B * kStepBytes, j);
  };
  const int steps = static_cast<int>((p.rows + 63) / 64);
  f32x4 acc[T16][T16];
  multiply<T, kCols, kCols, B, B, 2, 2>(lds, 0, steps, mrow, ncol, ncol + HALF / 2, at_step, issue, [](char*) {}, acc);
  uint16_t* out = second ? p.dwu : p.dwg;
#pragma unroll
  for (int j = 0; j < T16; ++j) {
    const int64_t m = f0 + row_of(mrow, j);
    if (m >= p.f) continue;
#pragma unroll
    for (int q = 0; q < T16 / 2; ++q) {
      const int n = n0 + ncol + 32 * q + 8 * (lane >> 4);
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
    gated_forward_kernel<T, 256><<<static_cast<unsigned>(t), 256, 0, stream>>>(p);
  else
    gated_forward_kernel<T, 128><<<static_cast<unsigned>(tiles(128, 128)), 256, 0, stream>>>(p);
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
      gated_dx_kernel<T, 256><<<p.tiles_m * p.tiles_n, 256, 0, stream>>>(p);
    } else {
      tiles(p.rows, p.d, 128);
      p.band = std::min(8, p.tiles_m);
      gated_dx_kernel<T, 128><<<p.tiles_m * p.tiles_n, 256, 0, stream>>>(p);
    }
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (p.dwg) {
    p.vec = wide(p.dwg, p.lddw) && wide(p.dwu, p.lddw);
    if (2 * tiles(p.f, p.d, 256) >= 200) {
      p.tiles_m *= 2;
      p.band = std::min(8, p.tiles_m);
      gated_dw_kernel<T, 256><<<p.tiles_m * p.tiles_n, 256, 0, stream>>>(p);
    } else {
      tiles(p.f, p.d, 128);
      p.tiles_m *= 2;
      p.band = std::min(8, p.tiles_m);
      gated_dw_kernel<T, 128><<<p.tiles_m * p.tiles_n, 256, 0, stream>>>(p);
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
