// Token embeddings: rows of a table by their numbers, and the table's gradient.
#include "layers_internal.h"
#include "vectors.h"

namespace opt8 {
namespace {

using namespace tile;

// Row `id` of a table of `rows`, or -1 where there is none.
template <class Id>
__device__ __forceinline__ int row_of(const void* ids, int64_t i, int64_t rows) {
  const int64_t id = static_cast<const Id*>(ids)[i];
  return id >= 0 && id < rows ? static_cast<int>(id) : -1;
}

// ---------------------------------------------------------------- lookup
struct Lookup {
  const void* ids;
  const void* table;
  const void* place_ids;
  const void* place_table;
  void* y;
  int64_t tokens, vocab, places, d, ldtable, ldplace, ldy;
  int64_t tasks;
  float scale;
  int column_blocks;
};

// A wave takes 512 columns of kTokens tokens, 8 columns to a lane; its rows are
// loaded before the first is stored.
constexpr int kTokens = 4;
template <class X, class Id>
__global__ __launch_bounds__(256) void lookup_kernel(const Lookup p) {
  const int64_t task = int64_t{blockIdx.x} * 4 + wave_id();
  if (task >= p.tasks) return;
  const int64_t first = task / p.column_blocks * kTokens;
  const int64_t c = task % p.column_blocks * 512 + (threadIdx.x & 63) * 8;
  const int64_t left = p.d - c;
  if (left <= 0) return;
  typedef typename Raw<X>::type Value;
  Eight<X> v[kTokens], at[kTokens];
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
    v[t].zero();
    at[t].zero();
    if (first + t >= p.tokens) continue;
    const int id = row_of<Id>(p.ids, first + t, p.vocab);
    if (id >= 0) v[t].load(static_cast<const Value*>(p.table) + id * p.ldtable + c, left);
    if (p.place_ids) {
      const int place = row_of<Id>(p.place_ids, first + t, p.places);
      if (place >= 0) at[t].load(static_cast<const Value*>(p.place_table) + place * p.ldplace + c, left);
    }
  }
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
    if (first + t >= p.tokens) continue;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = v[t][i] * p.scale;
      if (p.place_ids) y[i] += at[t][i];
    }
    store_eight<X>(static_cast<Value*>(p.y) + (first + t) * p.ldy + c, y, left);
  }
}

// ---------------------------------------------------------------- gradient
// The tokens sorted by id, those of one id by their place: a workgroup owns a range of
// ids and reads all of them twice, once to count and once to place.  Waves read
// consecutive stretches, and each has its own counter for every id, so that
// a token's position depends on the ids alone.
struct Sort {
  const void* ids;
  int64_t tokens, vocab;
  int range;
  int* order;     // token numbers
  int* keys;      // their ids
  int* starts;    // [vocab + 1], of each id's first
};

template <class Id>
__global__ __launch_bounds__(64 * kSortWaves) void sort_kernel(const Sort p) {
  constexpr int kThreads = 64 * kSortWaves, kUnroll = 8;
  __shared__ int count[kSortRange * kSortWaves];    // [id of the range][wave]
  __shared__ int sums[kSortWaves], belows[kSortWaves];
  const int t = threadIdx.x, lane = t & 63, wave = wave_id();
  const int low = static_cast<int>(blockIdx.x) * p.range;
  const int range = min(p.range, static_cast<int>(p.vocab) - low);
  for (int i = t; i < range * kSortWaves; i += kThreads) count[i] = 0;
  __syncthreads();

  const int64_t each = (p.tokens + kSortWaves * 64 - 1) / (kSortWaves * 64) * 64;
  const int64_t begin = wave * each, end = begin + each < p.tokens ? begin + each : p.tokens;
  int below = 0;
  for (int64_t i0 = begin; i0 < end; i0 += 64 * kUnroll) {
    int id[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + 64 * u + lane;
      id[u] = i < end ? row_of<Id>(p.ids, i, p.vocab) : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (id[u] >= 0 && id[u] < low) ++below;
      if (id[u] >= low && id[u] < low + range) atomicAdd(&count[(id[u] - low) * kSortWaves + wave], 1);
    }
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) below += __shfl_xor(below, s);
  if (lane == 0) belows[wave] = below;
  __syncthreads();

  // Exclusive sums over the counters, id by id and wave by wave: a thread's stretch, the
  // wave's threads, the waves.
  const int stretch = (range * kSortWaves + kThreads - 1) / kThreads;
  const int from = min(t * stretch, range * kSortWaves), to = min(from + stretch, range * kSortWaves);
  int mine = 0;
  for (int i = from; i < to; ++i) mine += count[i];
  int before = mine;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int other = __shfl_up(before, s);
    if (lane >= s) before += other;
  }
  if (lane == 63) sums[wave] = before;
  __syncthreads();
  int at = before - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    at += belows[w] + (w < wave ? sums[w] : 0);
    total += belows[w] + sums[w];
  }
  for (int i = from; i < to; ++i) {
    const int n = count[i];
    count[i] = at;
    if (i % kSortWaves == 0) p.starts[low + i / kSortWaves] = at;
    at += n;
  }
  if (t == 0 && low + range == p.vocab) p.starts[p.vocab] = total;
  __syncthreads();

  for (int64_t i0 = begin; i0 < end; i0 += 64 * kUnroll) {
    int id[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + 64 * u + lane;
      id[u] = i < end ? row_of<Id>(p.ids, i, p.vocab) : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      uint64_t open = __ballot(id[u] >= low && id[u] < low + range);
      while (open) {      // the ids among these 64, each once
        const int one = __builtin_amdgcn_readlane(id[u], __builtin_ctzll(open));
        const uint64_t same = __ballot(id[u] == one);
        int* next = &count[(one - low) * kSortWaves + wave];
        const int first = *next;
        if (id[u] == one) {
          const int to_ = first + __builtin_popcountll(same & ((uint64_t{1} << lane) - 1));
          p.order[to_] = static_cast<int>(i0 + 64 * u + lane);
          p.keys[to_] = one;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (lane == 0) *next = first + __builtin_popcountll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        open &= ~same;
      }
    }
  }
}

struct Sum {
  const int* order;
  const int* keys;
  const int* starts;
  const void* dy;
  void* dtable;
  float* partial;    // [chunk][2][d]
  int64_t vocab, d, lddy, lddtable;
  int64_t tasks;           // chunks * column blocks
  int64_t sum_groups;      // workgroups that add; those behind them store zeros
  float scale;
  int column_blocks, chunk, accumulate;
};

// 8 columns of one row of the gradient.
template <class D>
__device__ __forceinline__ void finish(const Sum& p, int id, int64_t c, int64_t left, float* sum) {
  auto* out = static_cast<typename Raw<D>::type*>(p.dtable) + id * p.lddtable + c;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] *= p.scale;
  if (p.accumulate) {
    Eight<D> old;
    old.load(out, left);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += old[i];
  }
  store_eight<D>(out, sum, left);
}

// A wave adds the rows of one chunk of sorted tokens, 512 columns of them, and gives
// each id's sum to the gradient, or, where an id goes on in another chunk, to the
// partial sums.  Chunks have the same number of tokens whatever their ids: one id
// with half of the tokens costs no more than as many different ones.
template <class X, class D>
__global__ __launch_bounds__(256) void sum_kernel(const Sum p) {
  const int lane = threadIdx.x & 63;
  if (blockIdx.x >= p.sum_groups) {
    const int64_t id = (blockIdx.x - p.sum_groups) * 4 + wave_id();
    if (id >= p.vocab || p.starts[id] != p.starts[id + 1]) return;
    const float none[8] = {};
    auto* out = static_cast<typename Raw<D>::type*>(p.dtable) + id * p.lddtable;
    for (int64_t c = lane * 8; c < p.d; c += 512) store_eight<D>(out + c, none, p.d - c);
    return;
  }
  const int64_t task = int64_t{blockIdx.x} * 4 + wave_id();
  if (task >= p.tasks) return;
  const int64_t chunk = task / p.column_blocks;
  const int64_t c = task % p.column_blocks * 512 + lane * 8;
  const int64_t left = p.d - c;
  const int total = p.starts[p.vocab];
  const int p0 = static_cast<int>(chunk) * p.chunk, p1 = min(p0 + p.chunk, total);
  if (p0 >= total) return;
  // lane i: the id of sorted token p0 - 1 + i
  const int at = p0 - 1 + lane;
  const int key = at >= 0 && at <= p1 && at < total ? p.keys[at] : -1;
  const int token = at >= p0 && at < p1 ? p.order[at] : 0;
  const auto* dy = static_cast<const typename Raw<X>::type*>(p.dy) + c;

  bool shared = __builtin_amdgcn_readlane(key, 0) == __builtin_amdgcn_readlane(key, 1);
  float sum[8] = {};
  constexpr int kAhead = 8;
  for (int j0 = 0; j0 < p1 - p0; j0 += kAhead) {
    Eight<X> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      v[u].zero();
      const int64_t row = __builtin_amdgcn_readlane(token, min(j0 + u + 1, 63));
      if (j0 + u < p1 - p0 && left > 0) v[u].load(dy + row * p.lddy, left);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      if (j >= p1 - p0) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[u][i];
      const int id = __builtin_amdgcn_readlane(key, j + 1);
      const bool goes_on = id == __builtin_amdgcn_readlane(key, j + 2);
      if (goes_on && j + 1 < p1 - p0) continue;
      if (left > 0) {
        if (!shared && !goes_on) finish<D>(p, id, c, left, sum);
        else store_some(p.partial + (2 * chunk + (shared ? 0 : 1)) * p.d + c, sum, left);
      }
      shared = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    }
  }
}

// Adds the partial sums of the id that starts in a chunk and goes on behind it, in the
// order of the chunks, cut into four stretches: a workgroup takes 1024 columns, 4 to a
// lane, its waves 256 columns of a stretch each.
template <class D>
__global__ __launch_bounds__(1024) void join_kernel(const Sum p) {
  __shared__ f32x4 parts[4][256];
  const int64_t blocks = (p.d + 1023) / 1024;
  const int chunk = static_cast<int>(blockIdx.x / blocks);
  const int total = p.starts[p.vocab];
  const int p0 = chunk * p.chunk, p1 = p0 + p.chunk;
  if (p1 >= total) return;
  const int id = p.keys[p1 - 1];
  const int first = p.starts[id], last = p.starts[id + 1];
  if (last <= p1 || first < p0) return;
  const int chunks = (last - 1) / p.chunk - chunk + 1;      // at least two
  const int lane = threadIdx.x & 63, wave = wave_id(), cut = wave >> 2;
  const int64_t c = blockIdx.x % blocks * 1024 + (wave & 3) * 256 + lane * 4;
  const int each = (chunks + 3) / 4;
  const int from = cut * each, to = min(from + each, chunks);
  const int count = static_cast<int>(p.d - c < 4 ? p.d - c : 4);
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* at = p.partial + 2 * int64_t{chunk} * p.d + c;
  if (count == 4) {
#pragma unroll 8
    for (int k = from; k < to; ++k) sum += *reinterpret_cast<const f32x4_at4*>(at + (k == 0 ? 1 : 2 * int64_t{k}) * p.d);
  } else {
    for (int k = from; k < to; ++k)
      for (int i = 0; i < 3; ++i)
        if (i < count) sum[i] += at[(k == 0 ? 1 : 2 * int64_t{k}) * p.d + i];
  }
  parts[cut][threadIdx.x & 255] = sum;
  __syncthreads();
  // 8 columns to a thread of the first two waves
  const int t = threadIdx.x;
  const int64_t c8 = blockIdx.x % blocks * 1024 + t * 8;
  if (t >= 128 || c8 >= p.d) return;
  float out[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    out[i] = parts[0][2 * t + i / 4][i % 4];
#pragma unroll
    for (int s = 1; s < 4; ++s) out[i] += parts[s][2 * t + i / 4][i % 4];
  }
  finish<D>(p, id, c8, p.d - c8, out);
}

template <class X>
hipError_t launch_lookup(Lookup& p, int id_type, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(pieces_of(p.tasks, 4));
  return id_type == OPT8_ID_INT32 ? queue(lookup_kernel<X, int32_t>, grid, 256, stream, p)
                                  : queue(lookup_kernel<X, int64_t>, grid, 256, stream, p);
}

template <class X, class D>
hipError_t launch_sums(Sum& p, int64_t chunks, hipStream_t stream) {
  const int64_t zero_groups = p.accumulate ? 0 : pieces_of(p.vocab, 4);
  hipError_t e = hipSuccess;
  if (p.sum_groups + zero_groups > 0)
    e = queue(sum_kernel<X, D>, static_cast<unsigned>(p.sum_groups + zero_groups), 256, stream, p);
  if (e == hipSuccess && chunks > 1)
    e = queue(join_kernel<D>, static_cast<unsigned>((chunks - 1) * pieces_of(p.d, 1024)), 1024, stream, p);
  return e;
}

}  // namespace

hipError_t launch_embedding_forward(const opt8_embedding& a, hipStream_t stream) {
  Lookup p;
  p.ids = a.ids;
  p.table = a.table;
  p.place_ids = a.place_ids;
  p.place_table = a.place_table;
  p.y = a.y;
  p.tokens = a.tokens;
  p.vocab = a.vocab;
  p.places = a.places;
  p.d = a.d;
  p.ldtable = a.ldtable;
  p.ldplace = a.ldplace;
  p.ldy = a.ldy;
  p.scale = a.scale;
  p.column_blocks = static_cast<int>(pieces_of(a.d, 512));
  p.tasks = pieces_of(a.tokens, kTokens) * p.column_blocks;
  if (a.type == OPT8_TYPE_BF16) return launch_lookup<Bf16>(p, a.id_type, stream);
  if (a.type == OPT8_TYPE_FP16) return launch_lookup<Fp16>(p, a.id_type, stream);
  return launch_lookup<float>(p, a.id_type, stream);
}

hipError_t launch_embedding_backward(const opt8_embedding_grad& a, hipStream_t stream) {
  const EmbeddingSpace space = embedding_space(a.tokens, a.vocab, a.d);
  char* work = static_cast<char*>(a.workspace);
  Sort s;
  s.ids = a.ids;
  s.tokens = a.tokens;
  s.vocab = a.vocab;
  s.range = static_cast<int>(sort_range(a.vocab));
  s.order = reinterpret_cast<int*>(work + space.order);
  s.keys = reinterpret_cast<int*>(work + space.keys);
  s.starts = reinterpret_cast<int*>(work + space.starts);
  const unsigned groups = static_cast<unsigned>(pieces_of(a.vocab, s.range));
  const hipError_t e = a.id_type == OPT8_ID_INT32 ? queue(sort_kernel<int32_t>, groups, 64 * kSortWaves, stream, s)
                                                  : queue(sort_kernel<int64_t>, groups, 64 * kSortWaves, stream, s);
  if (e != hipSuccess) return e;
  Sum p;
  p.order = s.order;
  p.keys = s.keys;
  p.starts = s.starts;
  p.dy = a.dy;
  p.dtable = a.dtable;
  p.partial = reinterpret_cast<float*>(work + space.partial);
  p.vocab = a.vocab;
  p.d = a.d;
  p.lddy = a.lddy;
  p.lddtable = a.lddtable;
  p.scale = a.scale;
  p.accumulate = a.accumulate != 0;
  p.chunk = static_cast<int>(sum_chunk(a.tokens, a.d));
  p.column_blocks = static_cast<int>(pieces_of(a.d, 512));
  const int64_t chunks = pieces_of(a.tokens, p.chunk);
  p.tasks = chunks * p.column_blocks;
  p.sum_groups = pieces_of(p.tasks, 4);
  const bool wide = a.dtable_type == OPT8_TYPE_FP32;
  if (a.type == OPT8_TYPE_BF16) return wide ? launch_sums<Bf16, float>(p, chunks, stream) : launch_sums<Bf16, Bf16>(p, chunks, stream);
  if (a.type == OPT8_TYPE_FP16) return wide ? launch_sums<Fp16, float>(p, chunks, stream) : launch_sums<Fp16, Fp16>(p, chunks, stream);
  return launch_sums<float, float>(p, chunks, stream);
}

}  // namespace opt8
