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
// exp by the hardware's base-2 exponential (2^-23.5 relative) of x*log2(e), whose
// rounding to fp32 adds |x| 2^-24: measured 2^-23 for |x| < 1, 2^-21 to 8, 2^-19 to 24
// and 2^-18 at the end of the range, far below a 16-bit result's half step.
// sigmoid(-inf) = 0 and sigmoid(inf) = 1.
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
    // Phi(-x) = phi(x) R(x) for x >= 0.  Mills' ratio R is smooth in t = 1/(1 +
    // 0.285 x): R = t * (a polynomial of degree 8 in t), minimax by reweighted least
    // squares on [0, inf), 1.6e-7 relative, 5e-7 in fp32.  About 14 instructions
    // where erfcf takes 60 (8192 x 16384 results: 59 us more than silu, against 255).
    const float x = __builtin_fabsf(g);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.285f, x, 1.0f));
    float r = 0.0615863354f;
    r = __builtin_fmaf(r, t, -0.21705334f);
    r = __builtin_fmaf(r, t, 0.18528194f);
    r = __builtin_fmaf(r, t, 0.00877245621f);
    r = __builtin_fmaf(r, t, 0.169393168f);
    r = __builtin_fmaf(r, t, 0.213377772f);
    r = __builtin_fmaf(r, t, 0.261955982f);
    r = __builtin_fmaf(r, t, 0.285000067f);
    r = __builtin_fmaf(r, t, 0.284999955f);
    const float density = 0.39894228040143268f * exp_fast(-0.5f * g * g);
    const float tail = density * r * t;
    const float below = g < 0.0f ? tail : 1.0f - tail;
    value = g * below;
    slope = __builtin_fmaf(g, density, below);
  } else {
    const float y = kTanhA * g * __builtin_fmaf(kTanhB * g, g, 1.0f);
    const float p = sigmoid(2.0f * y);
    value = g * p;
    // the bound keeps g*g finite beside the p(1 - p) = 0 of gates past 1e19
    const float dy2 = __builtin_fminf(2.0f * kTanhA * __builtin_fmaf(3.0f * kTanhB * g, g, 1.0f), 0x1p127f);
    slope = __builtin_fmaf(g * p * (1.0f - p), dy2, p);
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
};

// A tile holds B/2 rows of Wg and the same rows of Wu beside B rows of x; a
// wave takes as many columns of one as of the other, so g and u of one h meet
// in one lane.  8192 rows, d 4096, f 16384: 1.54 ms, with both projections stored
// 1.66 (1.33 PFLOP/s); about 10 us of a tile's 100 are its epilogue.  (The 256 x 256
// bf16 kernel spills 4 registers, outside the step loop.)
template <class T, class G>
__global__ __launch_bounds__(G::kThreads, G::kMinWaves) void gated_forward_kernel(const Forward p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int S = G::kSize, KG = G::kTeams, HALF = S / 2;
  __shared__ __align__(16) typename G::Lds lds;
  int tm, tn;
  tile_of_group(p.tiles_m, p.tiles_n, p.band, tm, tn);
  const int team = wave_id() / G::NW, wave = wave_id() % G::NW;
  const int mrow = wave / G::WN * (S / G::WM), ncol = wave % G::WN * (HALF / G::WN);
  const int m0 = tm * S, f0 = tn * HALF;
  const int kbytes = 2 * p.d;
  const int64_t kround = (kbytes + 15) & ~15;
  Loader<kRows, S, G::NW> la;
  Loader<kRows, HALF, G::NW / 2> lb;
  la.init(p.x + m0 * p.ldx, p.ldx, (std::min(S, p.rows - m0) - 1) * p.ldx + kround, 0, wave);
  const bool second = wave >= G::NW / 2;
  lb.init((second ? p.wu : p.wg) + f0 * p.ldw, p.ldw, (std::min(HALF, p.f - f0) - 1) * p.ldw + kround, 0,
          second ? wave - G::NW / 2 : wave);
  const int bto = (S + (second ? HALF : 0)) * kStepBytes;
  const int all_steps = (kbytes + kStepBytes - 1) / kStepBytes, steps = (all_steps + KG - 1) / KG;
  auto at_step = [&](int s) {
    const int step = s * KG + team;
    la.at_step(step, kbytes - step * kStepBytes);
    lb.at_step(step, kbytes - step * kStepBytes);
  };
  auto issue = [&](int j, uint32_t to, int i) {
    if (i == 0) la.issue(to, j);
    else lb.issue(to + bto, j);
  };
  auto last = [&](char* t) {
    if (kbytes & 15) {
      if (KG == 1 || (steps - 1) * KG + team + 1 == all_steps)
        clear_part_chunk<2 * S, 64 * G::NW>(t, kbytes - (all_steps - 1) * kStepBytes, threadIdx.x - team * 64 * G::NW);
      __syncthreads();
    }
  };
  f32x4 acc[G::MT][G::NT];
  multiply<T, G, kRows, kRows>(lds[team], steps, mrow, ncol, HALF + ncol, at_step, issue, last, acc);
  add_teams<KG, G::NW>(lds, team, wave, acc);

  constexpr int NG = G::NT / 4;       // 32-column groups of h in the wave's part
  constexpr int NS = KG == 1 ? NG : 1;    // of them stored together
  char* scratch = lds[0][0] + (team * G::NW + wave) * kRowScratch<NS>;
  __syncthreads();       // other waves may still read what the results are staged in
  with_act(p.act, [&](auto act) {
#pragma unroll
    for (int j = 0; j < G::MT; ++j)
#pragma unroll
      for (int q = 0; q < NG; q += NS) {
        if (KG > 1 && (j * NG + q) % KG != team) continue;    // each team its share
        const int n = f0 + ncol + 32 * q;
        if (n >= p.f) continue;
        float g[NS][8], u[NS][8], h[NS][8];
#pragma unroll
        for (int t = 0; t < NS; ++t) {
          take8(acc, q + t, j, g[t]);
          take8(acc, q + t + NG, j, u[t]);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[t][i] = activate<decltype(act)::value>(g[t][i]) * u[t][i];
        }
        store_rows<T, NS>(scratch, p.h + n, p.ldh, p.rows, p.f - n, m0, mrow, j, h);
        if (p.gate) {
          store_rows<T, NS>(scratch, p.gate + n, p.ldg, p.rows, p.f - n, m0, mrow, j, g);
          store_rows<T, NS>(scratch, p.up + n, p.ldg, p.rows, p.f - n, m0, mrow, j, u);
        }
      }
  });
#endif
}

// At most 16 rows (single tokens): the time is that of reading both weights, so
// nothing goes through LDS.  A workgroup owns 16 columns of h; each of its 4
// waves takes a quarter of k, in one piece (waves in turn would read all rows at
// one place of k at a time: where rows lie a power of two apart that is one memory
// channel), and adds its sums to the others' in a fixed order.  One row, d 4096, f
// 16384: 50 us, 268 MB at 5.4 TB/s.
__device__ __forceinline__ i32x4 load_part(const char* row, int at, int bytes) {
  i32x4 v = i32x4{0, 0, 0, 0};
  if (at < bytes) v = *reinterpret_cast<const i32x4*>(row + at);
  if (at + 16 > bytes) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int n = bytes - at - 4 * w;      // even
      if (n <= 0) v[w] = 0;
      else if (n < 4) v[w] &= 0xffff;
    }
  }
  return v;
}

template <class T>
__global__ __launch_bounds__(256) void gated_forward_few_kernel(const Forward p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kDepth = 4;
  __shared__ __align__(16) f32x4 sums[4][2][64];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16, bytes = 2 * p.d;
  const int64_t row = std::min(n0 + r, p.f - 1);
  const char* from[3] = {p.wg + row * p.ldw + g * 32, p.wu + row * p.ldw + g * 32,
                         p.x + std::min(r, p.rows - 1) * p.ldx + g * 32};
  f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
  struct Part {
    i32x4 v[3][2];
  };
  auto load = [&](Part& x, int step) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) x.v[i][h] = *reinterpret_cast<const i32x4*>(from[i] + step * kStepBytes + 16 * h);
  };
  auto add = [&](const Part& x) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      acc[0] = mfma16<T>(x.v[0][h], x.v[2][h], acc[0]);
      acc[1] = mfma16<T>(x.v[1][h], x.v[2][h], acc[1]);
    }
  };
  const int steps = bytes / kStepBytes;
  int step = steps * wave / 4;
  const int end = steps * (wave + 1) / 4;
  for (; step + kDepth <= end; step += kDepth) {
    Part x[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth; ++i) load(x[i], step + i);
#pragma unroll
    for (int i = 0; i < kDepth; ++i) add(x[i]);
  }
  for (; step < end; ++step) {
    Part x;
    load(x, step);
    add(x);
  }
  if (wave == 3 && bytes % kStepBytes) {
    Part x;
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) x.v[i][h] = load_part(from[i] + steps * kStepBytes, 16 * h, bytes % kStepBytes - g * 32);
    add(x);
  }
  sums[wave][0][lane] = acc[0];
  sums[wave][1][lane] = acc[1];
  __syncthreads();
  if (wave == 0 && r < p.rows) {
    f32x4 t[2];
#pragma unroll
    for (int w = 0; w < 2; ++w)
      t[w] = (sums[0][w][lane] + sums[1][w][lane]) + (sums[2][w][lane] + sums[3][w][lane]);
    const int64_t m = r;
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
#endif
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
  float* parts;         // dx before the last sum, [splits][rows][d]
  int splits;           // parts that dx's k is cut into
  int64_t rows, width;  // width: f rounded up to 64
  int64_t ldx, ldw;     // bytes
  int64_t lddh, ldg, lddx, lddw;
  int d, f, act;
  int tiles_m, tiles_n, band;
};

// dh * slope * up.  dh meets the slope first, so that a slope of 0 stays 0 where dh * up
// overflows; where their product leaves fp32's normal numbers (bf16 gradients do with
// saturated gates) the slope meets up instead, halved so that its 1.13 cannot overflow.
__device__ __forceinline__ float slope_product(float dh, float slope, float up) {
  const float first = dh * slope;
  return __builtin_fabsf(first) < 0x1p-126f ? 0.5f * slope * up * dh * 2.0f : first * up;
}

// dg and du, rounded to the type that the products take, zeros in the columns
// from f to width; 8 columns a thread.  8192 x 16384: 215 us, 1.34 GB at 6.2 TB/s.
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
        dg[i] = slope_product(dh, slope, value_of<T>(static_cast<uint16_t>(rc[i])));
        du[i] = dh * value;
      }
    });
    uint16_t* o = reinterpret_cast<uint16_t*>(p.both) + m * 2 * p.width + n;
    *reinterpret_cast<i32x4*>(o) = packed<T>(dg);
    *reinterpret_cast<i32x4*>(o + p.width) = packed<T>(du);
  }
}

// The wave's sums to rows m0 + mrow.. and columns n0.. of a [rows, cols] matrix;
// of several teams each stores its share.
template <class T, class G, class Out>
__device__ __forceinline__ void store_tile(char* copies, Out* out, int64_t ld, int64_t rows, int cols, int64_t m0, int mrow,
                                           int n0, int team, int wave, const f32x4 (&acc)[G::MT][G::NT]) {
  constexpr int NG = G::NT / 2, KG = G::kTeams, NS = KG == 1 ? NG : 1;
  char* scratch = copies + (team * G::NW + wave) * kRowScratch<NS>;
  __syncthreads();       // other waves may still read what the results are staged in
#pragma unroll
  for (int j = 0; j < G::MT; ++j)
#pragma unroll
    for (int q = 0; q < NG; q += NS) {
      if (KG > 1 && (j * NG + q) % KG != team) continue;
      const int n = n0 + 32 * q;
      if (n >= cols) continue;
      if constexpr (std::is_same<T, float>::value) {
        const int64_t m = m0 + row_of(mrow, j);
        const int at = n + 8 * ((threadIdx.x & 63) >> 4);
#pragma unroll
        for (int t = 0; t < NS; ++t) {
          float v[8];
          take8(acc, q + t, j, v);
          if (m < rows) store_some(out + m * ld + at + 32 * t, v, cols - at - 32 * t);
        }
      } else {
        float v[NS][8];
#pragma unroll
        for (int t = 0; t < NS; ++t) take8(acc, q + t, j, v[t]);
        store_rows<T, NS>(scratch, out + n, ld, rows, cols - n, m0, mrow, j, v);
      }
    }
}

// dx = [dg du] [Wg; Wu]: k runs along the rows of the weights.  (The 256 x 256 kernel
// spills 20 registers, outside the step loop.)
template <class T, class G>
__global__ __launch_bounds__(G::kThreads, G::kMinWaves) void gated_dx_kernel(const Backward p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int S = G::kSize, KG = G::kTeams;
  __shared__ __align__(16) typename G::Lds lds;
  int tm, tn;
  tile_of_group(p.tiles_m, p.tiles_n, p.band, tm, tn);
  const int team = wave_id() / G::NW, wave = wave_id() % G::NW;
  const int mrow = wave / G::WN * (S / G::WM), ncol = wave % G::WN * (S / G::WN);
  const int64_t m0 = int64_t{tm} * S;
  const int n0 = tn * S;
  const int64_t lda = 4 * p.width;
  Loader<kRows, S, G::NW> la;
  Loader<kCols, S, G::NW> lb;
  la.init(p.both + m0 * lda, lda, std::min<int64_t>(S, p.rows - m0) * lda, 0, wave);
  lb.init(p.wg + 2 * n0, p.ldw, (p.f - 1) * p.ldw + ((2 * int64_t{p.d} + 15) & ~int64_t{15}) - 2 * n0, p.d - n0, wave);
  // blockIdx.y: the part of k
  const int half = static_cast<int>(p.width / 64), per = (2 * half + p.splits - 1) / p.splits;
  const int begin = blockIdx.y * per, end = std::min(2 * half, begin + per), steps = (end - begin + KG - 1) / KG;
  auto at_step = [&](int s) {
    const int step = begin + s * KG + team;
    la.at_step(step, (end - step) * kStepBytes);
    lb.base = (step < half ? p.wg : p.wu) + 2 * n0;
    lb.at_step(step >= end ? 2 * half : step < half ? step : step - half, 0);
  };
  auto issue = [&](int j, uint32_t to, int i) {
    if (i == 0) la.issue(to, j);
    else lb.issue(to + S * kStepBytes, j);
  };
  f32x4 acc[G::MT][G::NT];
  multiply<T, G, kRows, kCols>(lds[team], steps, mrow, ncol, ncol + S / G::WN / 2, at_step, issue, [](char*) {}, acc);
  add_teams<KG, G::NW>(lds, team, wave, acc);
  if (p.splits == 1)
    store_tile<T, G>(lds[0][0], p.dx, p.lddx, p.rows, p.d, m0, mrow, n0 + ncol, team, wave, acc);
  else
    store_tile<float, G>(lds[0][0], p.parts + blockIdx.y * p.rows * p.d, p.d, p.rows, p.d, m0, mrow, n0 + ncol, team, wave, acc);
#endif
}

// dx from its parts, added in their order.
template <class T>
__global__ __launch_bounds__(256) void gated_dx_sum_kernel(const Backward p) {
  const int64_t total = p.rows * p.d;
  for (int64_t at = int64_t{blockIdx.x} * 256 + threadIdx.x; at < total; at += int64_t{gridDim.x} * 256) {
    float v = p.parts[at];
    for (int i = 1; i < p.splits; ++i) v += p.parts[i * total + at];
    p.dx[at / p.d * p.lddx + at % p.d] = static_cast<uint16_t>(bits_of(T{}, v));
  }
}

// dWg = dg^T x and dWu = du^T x: k is the rows (tokens) of both operands.
template <class T, class G>
__global__ __launch_bounds__(G::kThreads, G::kMinWaves) void gated_dw_kernel(const Backward p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int S = G::kSize, KG = G::kTeams;
  __shared__ __align__(16) typename G::Lds lds;
  int tm, tn;
  tile_of_group(p.tiles_m, p.tiles_n, p.band, tm, tn);
  const int team = wave_id() / G::NW, wave = wave_id() % G::NW;
  const int mrow = wave / G::WN * (S / G::WM), ncol = wave % G::WN * (S / G::WN);
  const int one = p.tiles_m / 2;
  const bool second = tm >= one;
  const int f0 = (second ? tm - one : tm) * S, n0 = tn * S;
  const int64_t lda = 4 * p.width;
  Loader<kCols, S, G::NW> la, lb;
  const int64_t off = 2 * (f0 + (second ? p.width : 0));
  la.init(p.both + off, lda, p.rows * lda - off, static_cast<int>(p.width) - f0, wave);
  lb.init(p.x + 2 * n0, p.ldx, (p.rows - 1) * p.ldx + ((2 * int64_t{p.d} + 15) & ~int64_t{15}) - 2 * n0, p.d - n0, wave);
  auto at_step = [&](int s) {
    la.at_step(s * KG + team, 0);
    lb.at_step(s * KG + team, 0);
  };
  auto issue = [&](int j, uint32_t to, int i) {
    if (i == 0) la.issue(to, j);
    else lb.issue(to + S * kStepBytes, j);
  };
  const int steps = static_cast<int>((p.rows + 64 * KG - 1) / (64 * KG));
  f32x4 acc[G::MT][G::NT];
  multiply<T, G, kCols, kCols>(lds[team], steps, mrow, ncol, ncol + S / G::WN / 2, at_step, issue, [](char*) {}, acc);
  add_teams<KG, G::NW>(lds, team, wave, acc);
  store_tile<T, G>(lds[0][0], second ? p.dwu : p.dwg, p.lddw, p.f, p.d, f0, mrow, n0 + ncol, team, wave, acc);
#endif
}

// Calls f with the chosen tiling.
template <class F>
void with_tiling(int choice, F&& f) {
  switch (choice) {
    case kTile256: return f(Tiling<256, 1>{});
    case kTile128: return f(Tiling<128, 1>{});
    case kTile128Teams2: return f(Tiling<128, 2>{});
    case kTile64Teams2: return f(Tiling<64, 2>{});
    default: return f(Tiling<64, 4>{});
  }
}

template <class T>
hipError_t forward(Forward& p, hipStream_t stream) {
  if (p.rows <= kFewRows) return queue(gated_forward_few_kernel<T>, (p.f + 15) / 16, 256, stream, p);
  hipError_t e = hipSuccess;
  with_tiling(gated_forward_choice(p.rows, p.d, p.f), [&](auto g) {
    typedef decltype(g) G;
    p.tiles_m = (p.rows + G::kSize - 1) / G::kSize;
    p.tiles_n = (p.f + G::kSize / 2 - 1) / (G::kSize / 2);
    p.band = std::min(8, p.tiles_m);
    e = queue(gated_forward_kernel<T, G>, p.tiles_m * p.tiles_n, G::kThreads, stream, p);
  });
  return e;
}

template <class T>
hipError_t backward(Backward& p, hipStream_t stream) {
  hipError_t e = hipSuccess;
  const int64_t chunks = p.rows * (p.width / 8);
  if (chunks > 0) {
    e = queue(gated_slopes_kernel<T>, static_cast<unsigned>(std::min<int64_t>((chunks + 255) / 256, 1 << 20)), 256, stream, p);
    if (e != hipSuccess) return e;
  }
  auto cover = [&](int64_t m, int64_t n, int size) {
    p.tiles_m = static_cast<int>((m + size - 1) / size);
    p.tiles_n = static_cast<int>((n + size - 1) / size);
  };
  if (p.dx && p.rows > 0) {
    with_tiling(gated_dx_choice(p.rows, p.d, p.f), [&](auto g) {
      typedef decltype(g) G;
      cover(p.rows, p.d, G::kSize);
      p.band = std::min(8, p.tiles_m);
      e = queue(gated_dx_kernel<T, G>, dim3(p.tiles_m * p.tiles_n, p.splits), G::kThreads, stream, p);
    });
    if (e != hipSuccess) return e;
    if (p.splits > 1) {
      e = queue(gated_dx_sum_kernel<T>, static_cast<unsigned>((p.rows * p.d + 255) / 256), 256, stream, p);
      if (e != hipSuccess) return e;
    }
  }
  if (p.dwg) {
    with_tiling(gated_dw_choice(p.rows, p.d, p.f), [&](auto g) {
      typedef decltype(g) G;
      cover(p.f, p.d, G::kSize);
      p.tiles_m *= 2;
      p.band = std::min(8, p.tiles_m);
      e = queue(gated_dw_kernel<T, G>, p.tiles_m * p.tiles_n, G::kThreads, stream, p);
    });
  }
  return e;
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
  p.parts = reinterpret_cast<float*>(p.both + gated_bytes(a.rows, a.f));
  p.splits = gated_dx_splits(a.rows, a.d, a.f);
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
  return a.type == OPT8_TYPE_BF16 ? backward<Bf16>(p, stream) : backward<Fp16>(p, stream);
}

}  // namespace opt8
