// Norm of a list of gradients, and their clipping.
#include <algorithm>

#include "layers_internal.h"
#include "vectors.h"

namespace opt8 {
namespace {

using namespace tile;

constexpr int kThreads = 256;
constexpr int kPasses = OPT8_GRAD_PIECE / (kThreads * 8);    // 8 values to a thread in each

// The head's pieces, and no more than the table has room for: a table may be larger than
// its list's, and what lies behind the list's pieces is not one.
__device__ __forceinline__ int64_t pieces_there(const GradPiece* pieces, int64_t room) {
  const int64_t listed = reinterpret_cast<const GradHead*>(pieces - 1)->pieces;
  return listed < room ? listed : room;
}

struct NormOf {
  const GradPiece* pieces;    // behind the table's head
  int64_t room;
  double* sums;       // [groups]
  double* squares;
  float* norm;
  int groups;
  int stream;
};

// Sum over a workgroup, in its first thread.
__device__ __forceinline__ double sum_of_group(double x) {
  __shared__ double waves[kThreads / 64];
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) x += __shfl_xor(x, s);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = x;
  __syncthreads();
  x = waves[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) x += waves[w];
  return x;
}

// Squares in 64 bits: exact, and no gradient's is too large or too small for them.
template <class X>
__device__ __forceinline__ void add_squares(const GradPiece& p, bool stream, double* sum) {
  const auto* from = static_cast<const typename Raw<X>::type*>(p.from);
  Eight<X> v[kPasses];
  if (stream && p.count == OPT8_GRAD_PIECE) {
#pragma unroll
    for (int k = 0; k < kPasses; ++k) v[k].stream(from + (k * kThreads + static_cast<int>(threadIdx.x)) * 8, 8);
  } else {
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int at = (k * kThreads + static_cast<int>(threadIdx.x)) * 8;
      v[k].zero();
      if (at < p.count) v[k].load(from + at, p.count - at);
    }
  }
#pragma unroll
  for (int k = 0; k < kPasses; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double x = static_cast<double>(v[k][i]);
      sum[i & 1] = __builtin_fma(x, x, sum[i & 1]);
    }
}

// Workgroups walk through the pieces; where the next one lies is read ahead.  Bound by
// memory: 2.65G bf16 values in 780 us (6.8 TB/s); squares in 32 bits would take 1.3% less.
__global__ __launch_bounds__(kThreads) void squares_kernel(const NormOf p) {
  double sum[2] = {0.0, 0.0};
  GradPiece next = p.pieces[blockIdx.x];
  const int64_t count = pieces_there(p.pieces, p.room);
  for (int64_t i = blockIdx.x; i < count; i += p.groups) {
    const GradPiece piece = next;
    if (i + p.groups < count) next = p.pieces[i + p.groups];
    if (piece.type == OPT8_TYPE_BF16) add_squares<Bf16>(piece, p.stream, sum);
    else if (piece.type == OPT8_TYPE_FP16) add_squares<Fp16>(piece, p.stream, sum);
    else add_squares<float>(piece, p.stream, sum);
  }
  const double all = sum_of_group(sum[0] + sum[1]);
  if (threadIdx.x == 0) p.sums[blockIdx.x] = all;
}

// The workgroups' sums, by one more.
__global__ __launch_bounds__(kThreads) void norm_kernel(const NormOf p) {
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < kGradGroups / kThreads; ++k) {
    const int i = k * kThreads + static_cast<int>(threadIdx.x);
    if (i < p.groups) sum += p.sums[i];
  }
  sum = sum_of_group(sum);
  if (threadIdx.x != 0) return;
  *p.squares = sum;
  if (p.norm) *p.norm = static_cast<float>(__builtin_sqrt(sum));
}

struct Clip {
  const GradPiece* pieces;    // behind the table's head
  int64_t room;
  const double* squares;
  float* norm;
  double max_norm;
  int groups;
};

template <class X, class Y>
__device__ __forceinline__ void scaled(const GradPiece& p, float factor) {
  const auto* from = static_cast<const typename Raw<X>::type*>(p.from);
  auto* to = static_cast<typename Raw<Y>::type*>(p.to);
  Eight<X> v[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int at = (k * kThreads + static_cast<int>(threadIdx.x)) * 8;
    v[k].zero();
    if (at < p.count) v[k].load(from + at, p.count - at);
  }
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int at = (k * kThreads + static_cast<int>(threadIdx.x)) * 8;
    float out[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = v[k][i] * factor;
    if (at < p.count) stream_eight<Y>(to + at, out, p.count - at);
  }
}

template <class X>
__device__ __forceinline__ void scaled_to(const GradPiece& p, float factor) {
  if (p.to_type == OPT8_TYPE_BF16) scaled<X, Bf16>(p, factor);
  else if (p.to_type == OPT8_TYPE_FP16) scaled<X, Fp16>(p, factor);
  else scaled<X, float>(p, factor);
}

// 355M fp32 values to bf16: 370 us for 2.1 GB (5.8 TB/s).  With a factor of 1 the list's
// pieces in place are not even looked up (324,000 of them: 4 us; looked up one by one 68).
__global__ __launch_bounds__(kThreads) void clip_kernel(const Clip p) {
  const double norm = __builtin_sqrt(*p.squares);
  if (p.norm && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = static_cast<float>(norm);
  const double ratio = p.max_norm / (norm + 1e-6);
  const float factor = ratio >= 1.0 ? 1.0f : static_cast<float>(ratio);    // NaN stays NaN
  // pieces with a place of their own come first: all that there is to do by a factor of 1
  const int64_t own = reinterpret_cast<const GradHead*>(p.pieces - 1)->own, all = pieces_there(p.pieces, p.room);
  const int64_t count = factor == 1.0f && own < all ? own : all;
  for (int64_t i = blockIdx.x; i < count; i += p.groups) {
    const GradPiece piece = p.pieces[i];
    if (piece.type == OPT8_TYPE_BF16) scaled_to<Bf16>(piece, factor);
    else if (piece.type == OPT8_TYPE_FP16) scaled_to<Fp16>(piece, factor);
    else scaled_to<float>(piece, factor);
  }
}

static_assert(kGradGroups * sizeof(double) <= OPT8_GRAD_WORKSPACE, "the workgroups' sums");
int groups_of(int64_t pieces) { return static_cast<int>(std::min<int64_t>(pieces, kGradGroups)); }

}  // namespace

hipError_t launch_grad_norm(const opt8_grads& a, hipStream_t stream) {
  NormOf p;
  p.pieces = static_cast<const GradPiece*>(a.table) + 1;
  p.room = a.table_bytes / OPT8_GRAD_PIECE_BYTES - 1;
  p.sums = static_cast<double*>(a.workspace);
  p.squares = a.squares;
  p.norm = a.norm;
  p.groups = groups_of(p.room);
  p.stream = streams(p.room * OPT8_GRAD_PIECE * 2);
  if (p.groups > 0) {
    const hipError_t e = queue(squares_kernel, static_cast<unsigned>(p.groups), kThreads, stream, p);
    if (e != hipSuccess) return e;
  }
  return queue(norm_kernel, 1, kThreads, stream, p);
}

hipError_t launch_grad_clip(const opt8_grads& a, hipStream_t stream) {
  Clip p;
  p.pieces = static_cast<const GradPiece*>(a.table) + 1;
  p.room = a.table_bytes / OPT8_GRAD_PIECE_BYTES - 1;
  p.squares = a.squares;
  p.norm = a.norm;
  p.max_norm = a.max_norm;
  p.groups = std::max(1, groups_of(p.room));
  return queue(clip_kernel, static_cast<unsigned>(p.groups), kThreads, stream, p);
}

}  // namespace opt8
