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

// A wave takes 512 columns of kTokens tokens, 8 columns to a lane.  One load brings the
// tokens' ids and one their places (a lane each), the next ones all rows.  Bound by
// memory: 16384 tokens of 4096 bf16 values with places 39 us, 256 MB of them read and
// written (rows of frequent ids once by each XCD's L2) at 6.6 TB/s; with one token to a
// wave 41, with four 39.6.
constexpr int kTokens = 2;
template <class X, class Id>
__global__ __launch_bounds__(256) void lookup_kernel(const Lookup p) {
  const int64_t task = int64_t{blockIdx.x} * 4 + wave_id();
  if (task >= p.tasks) return;
  const int lane = threadIdx.x & 63;
  const int64_t first = task / p.column_blocks * kTokens;
  const int64_t c = task % p.column_blocks * 512 + lane * 8;
  const int64_t left = p.d - c;
  typedef typename Raw<X>::type Value;
  const bool some = lane < kTokens && first + lane < p.tokens;
  const int ids = some ? row_of<Id>(p.ids, first + lane, p.vocab) : -1;
  const int places = some && p.place_ids ? row_of<Id>(p.place_ids, first + lane, p.places) : -1;
  Eight<X> v[kTokens], at[kTokens];
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
    v[t].zero();
    at[t].zero();
    const int64_t id = __builtin_amdgcn_readlane(ids, t), place = __builtin_amdgcn_readlane(places, t);
    if (id >= 0 && left > 0) v[t].load(static_cast<const Value*>(p.table) + id * p.ldtable + c, left);
    if (place >= 0 && left > 0) at[t].load(static_cast<const Value*>(p.place_table) + place * p.ldplace + c, left);
  }
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
    if (first + t >= p.tokens || left <= 0) break;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = v[t][i] * p.scale;
      if (p.place_ids) y[i] += at[t][i];
    }
    stream_eight<X>(static_cast<Value*>(p.y) + (first + t) * p.ldy + c, y, left);
  }
}

// ---------------------------------------------------------------- gradient
// An id is the (id / groups)-th of its workgroup's.  The workgroup is id modulo groups,
// moved on with every round: neither neighbours nor multiples of a power of two, which
// ids in use together often are, fall to one.
constexpr int kTurn = 37;
__device__ __forceinline__ int owner_of(int id, const SortShape& s) { return (id + (id >> s.shift) * kTurn) & (s.groups - 1); }
__device__ __forceinline__ int id_of(int owner, int own, const SortShape& s) { return own << s.shift | ((owner - own * kTurn) & (s.groups - 1)); }
// Where its tokens start among the sorted ones stands in starts[slot_of(id)], and where
// they end in the next place.
__device__ __forceinline__ int slot_of(int id, const SortShape& s) { return owner_of(id, s) * s.range + (id >> s.shift); }

// The tokens sorted by their id's slot, those of one id by their place: a workgroup
// owns a share of the ids and reads all tokens, counting its own ones and noting where
// they stand, and then gives them their positions.  Waves read consecutive stretches,
// and each has its own counter for every id, so that a token's position depends on the
// ids alone.  A wave that finds more than it can note (where one id has over 512 of its
// stretch's tokens) reads its stretch again.  256 workgroups read 16384 ids in 9.4
// to 11.5 us, 1001 in 6.0, 65536 in 28.7; with an adjacent range of ids to each, where a
// few workgroups have the frequent ones, 16384 took 94 and 1001 10.5.
struct Sort {
  const void* ids;
  int64_t tokens, vocab;
  SortShape shape;
  int* order;     // token numbers
  int* keys;      // their ids
  int* starts;    // [groups * range + 1]
};

template <class Id>
__global__ __launch_bounds__(64 * kSortWaves) void sort_kernel(const Sort p) {
  constexpr int kThreads = 64 * kSortWaves, kUnroll = 8, kNoted = 512;
  __shared__ int count[kSortRange * kSortWaves];    // [id of the workgroup][wave]
  __shared__ int noted[kSortWaves][kNoted];         // id of the workgroup << kPlaceBits | place in the wave's stretch
  __shared__ int sums[kSortWaves], belows[kSortWaves];
  constexpr int kPlaceBits = 19;
  static_assert(kSortRange <= 1 << (31 - kPlaceBits) && (1 << 22) / kSortWaves + 64 <= 1 << kPlaceBits, "a note's bits");
  const int t = threadIdx.x, lane = t & 63, wave = wave_id();
  const int group = static_cast<int>(blockIdx.x), range = p.shape.range;
  for (int i = t; i < range * kSortWaves; i += kThreads) count[i] = 0;
  __syncthreads();

  const int64_t each = (p.tokens + kThreads - 1) / kThreads * 64;
  const int64_t begin = wave * each, end = begin + each < p.tokens ? begin + each : p.tokens;
  const uint64_t under = (uint64_t{1} << lane) - 1;
  int below = 0, found = 0;
  for (int64_t i0 = begin; i0 < end; i0 += 64 * kUnroll) {
    int id[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + 64 * u + lane;
      id[u] = i < end ? row_of<Id>(p.ids, i, p.vocab) : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int owner = id[u] < 0 ? p.shape.groups : owner_of(id[u], p.shape);
      below += owner < group;
      const uint64_t mine = __ballot(owner == group);
      if (mine == 0) continue;
      if (owner == group) {
        const int own = id[u] >> p.shape.shift, at = found + __builtin_popcountll(mine & under);
        atomicAdd(&count[own * kSortWaves + wave], 1);
        if (at < kNoted) noted[wave][at] = own << kPlaceBits | static_cast<int>(i0 - begin + 64 * u + lane);
      }
      found += __builtin_popcountll(mine);
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
    if (i % kSortWaves == 0) p.starts[group * range + i / kSortWaves] = at;
    at += n;
  }
  if (t == 0 && group == p.shape.groups - 1) p.starts[p.shape.groups * range] = total;
  __syncthreads();

  // Positions for 64 tokens of the wave's, in their order: own < 0 where there is none.
  auto place = [&](int own, int64_t token) {
    uint64_t open = __ballot(own >= 0);
    while (open) {      // the ids among them, each once
      const int one = __builtin_amdgcn_readlane(own, __builtin_ctzll(open));
      const uint64_t same = __ballot(own == one);
      int* next = &count[one * kSortWaves + wave];
      const int first = *next;
      if (own == one) {
        const int to = first + __builtin_popcountll(same & under);
        p.order[to] = static_cast<int>(token);
        p.keys[to] = id_of(group, one, p.shape);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (lane == 0) *next = first + __builtin_popcountll(same);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      open &= ~same;
    }
  };
  if (found <= kNoted) {
    for (int i = lane; i - lane < found; i += 64) {
      const int note = i < found ? noted[wave][i] : -1;
      place(note < 0 ? -1 : note >> kPlaceBits, begin + (note & ((1 << kPlaceBits) - 1)));
    }
  } else {
    for (int64_t i0 = begin; i0 < end; i0 += 64) {
      const int64_t i = i0 + lane;
      const int id = i < end ? row_of<Id>(p.ids, i, p.vocab) : -1;
      place(id >= 0 && owner_of(id, p.shape) == group ? id >> p.shape.shift : -1, i);
    }
  }
}

struct Sum {
  const void* ids;
  const int* order;
  const int* keys;
  const int* starts;
  SortShape shape;
  const void* dy;
  void* dtable;
  float* partial;    // [chunk][2][d]
  int64_t tokens, vocab, d, lddy, lddtable;
  int64_t tasks;           // chunks (or tokens) * column blocks
  int64_t sum_groups;      // workgroups that add; those behind them store zeros
  float scale;
  int column_blocks, chunk, accumulate, stream;
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

// Zeros in 512 columns of one row, by a wave.
template <class D>
__device__ __forceinline__ void clear(void* dtable, int64_t row, int64_t block, int64_t d, int64_t ld) {
  const float none[8] = {};
  const int64_t c = block * 512 + (threadIdx.x & 63) * 8;
  if (c < d) stream_eight<D>(static_cast<typename Raw<D>::type*>(dtable) + row * ld + c, none, d - c);
}

// At most kFewTokens tokens, without a sort: a wave takes 512 columns of one token, holds
// all ids in its lanes, and if no token before its own has the same id, it adds the rows
// of all that have, in their order.  Waves behind those clear the rows without tokens
// (50257 x 4096 bf16 in 57 us with the call's launch, 7.2 TB/s).
template <class X, class D, class Id>
__global__ __launch_bounds__(256) void few_kernel(const Sum p) {
  static_assert(kFewTokens <= 128, "two ids to a lane");
  typedef typename Raw<X>::type Value;
  const int lane = threadIdx.x & 63;
  const int a = lane < p.tokens ? row_of<Id>(p.ids, lane, p.vocab) : -1;
  const int b = lane + 64 < p.tokens ? row_of<Id>(p.ids, lane + 64, p.vocab) : -1;
  int64_t task = int64_t{blockIdx.x} * 4 + wave_id();
  if (task >= p.tasks) {
    task -= p.tasks;
    const int64_t row = task / p.column_blocks;
    if (p.accumulate || row >= p.vocab || __ballot(a == row || b == row) != 0) return;
    clear<D>(p.dtable, row, task % p.column_blocks, p.d, p.lddtable);
    return;
  }
  const int token = static_cast<int>(task / p.column_blocks);
  const int64_t c = task % p.column_blocks * 512 + lane * 8, left = p.d - c;
  const int id = token < 64 ? __builtin_amdgcn_readlane(a, token) : __builtin_amdgcn_readlane(b, token - 64);
  if (id < 0) return;
  uint64_t low = __ballot(a == id), high = __ballot(b == id);
  if ((low ? __builtin_ctzll(low) : 64 + __builtin_ctzll(high)) != token) return;
  const Value* dy = static_cast<const Value*>(p.dy) + c;
  constexpr int kAhead = 8;
  float sum[8] = {};
  while (low | high) {
    Eight<X> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      v[u].zero();
      int64_t row = -1;
      if (low) {
        row = __builtin_ctzll(low);
        low &= low - 1;
      } else if (high) {
        row = 64 + __builtin_ctzll(high);
        high &= high - 1;
      }
      if (row >= 0 && left > 0) v[u].load(dy + row * p.lddy, left);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[u][i];
  }
  if (left > 0) finish<D>(p, id, c, left, sum);
}

// A wave adds the rows of one chunk of sorted tokens, 512 columns of them, and gives
// each id's sum to the gradient, or, where an id goes on in another chunk, to the
// partial sums.  Chunks have the same number of tokens whatever their ids: one id
// with half of the tokens costs no more than as many different ones.  Waves behind them
// clear the rows without tokens, 1 KB each in the order of the addresses (with a row of
// 8 KB to a wave the clearing runs at 5.5 TB/s instead of 6.7).  Bound by memory: 12288 of
// 16384 tokens into 50257 x 4096 bf16, 518 MB in 75 us (6.9 TB/s).
template <class X, class D>
__global__ __launch_bounds__(256) void sum_kernel(const Sum p) {
  const int lane = threadIdx.x & 63;
  if (blockIdx.x >= p.sum_groups) {
    const int64_t task = (blockIdx.x - p.sum_groups) * 4 + wave_id(), id = task / p.column_blocks;
    if (id >= p.vocab) return;
    const int slot = slot_of(static_cast<int>(id), p.shape);
    if (p.starts[slot] != p.starts[slot + 1]) return;
    clear<D>(p.dtable, id, task % p.column_blocks, p.d, p.lddtable);
    return;
  }
  const int64_t task = int64_t{blockIdx.x} * 4 + wave_id();
  if (task >= p.tasks) return;
  const int64_t chunk = task / p.column_blocks;
  const int64_t c = task % p.column_blocks * 512 + lane * 8;
  const int64_t left = p.d - c;
  const int total = p.starts[p.shape.groups * p.shape.range];
  const int p0 = static_cast<int>(chunk) * p.chunk, p1 = min(p0 + p.chunk, total);
  if (p0 >= total) return;
  // lane i: the id of sorted token p0 - 1 + i
  const int at = p0 - 1 + lane;
  const int key = at >= 0 && at <= p1 && at < total ? p.keys[at] : -1;
  const int token = at >= p0 && at < p1 ? p.order[at] : 0;
  typedef typename Raw<X>::type Value;
  const Value* dy = static_cast<const Value*>(p.dy) + c;

  bool shared = __builtin_amdgcn_readlane(key, 0) == __builtin_amdgcn_readlane(key, 1);
  float sum[8] = {};
  constexpr int kAhead = 8;
  for (int j0 = 0; j0 < p1 - p0; j0 += kAhead) {
    Eight<X> v[kAhead];
    auto read = [&](auto&& one) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        v[u].zero();
        const int64_t row = __builtin_amdgcn_readlane(token, min(j0 + u + 1, 63));
        if (j0 + u < p1 - p0 && left > 0) one(v[u], dy + row * p.lddy);
      }
    };
    if (p.stream) read([&](Eight<X>& to, const Value* at) { to.stream(at, left); });
    else read([&](Eight<X>& to, const Value* at) { to.load(at, left); });
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
// order of the chunks, cut into kCuts stretches: a workgroup takes 1024 columns, 4 to a
// lane, its waves 256 columns of a stretch each.  In 64 bits: 2^22 tokens of one id are
// 2^17 partial sums, and as many additions of like signs in 32 bits drift by thousands
// of roundings.  Mostly the time to find that there is little to do (7 us of the case
// above); with one, two and four stretches 65536 tokens of 1024 columns take 82.4, 81.0
// and 83.1 us in all, 16384 of 4096 columns and one id 80.5, 75.5 and 75.3, 1001 of 1600 17.5,
// 16.5 and 16.4.
constexpr int kCuts = 2;
typedef __attribute__((ext_vector_type(4))) double f64x4;
template <class D>
__global__ __launch_bounds__(256 * kCuts) void join_kernel(const Sum p) {
  __shared__ f64x4 parts[kCuts][256];
  const int64_t blocks = (p.d + 1023) / 1024;
  const int chunk = static_cast<int>(blockIdx.x / blocks);
  const int total = p.starts[p.shape.groups * p.shape.range];
  const int p0 = chunk * p.chunk, p1 = p0 + p.chunk;
  if (p1 >= total) return;
  const int id = p.keys[p1 - 1];
  const int slot = slot_of(id, p.shape);
  const int first = p.starts[slot], last = p.starts[slot + 1];
  if (last <= p1 || first < p0) return;
  const int chunks = (last - 1) / p.chunk - chunk + 1;      // at least two
  const int lane = threadIdx.x & 63, wave = wave_id(), cut = wave >> 2;
  const int64_t c = blockIdx.x % blocks * 1024 + (wave & 3) * 256 + lane * 4;
  const int each = (chunks + kCuts - 1) / kCuts;
  const int from = cut * each, to = min(from + each, chunks);
  const int count = static_cast<int>(p.d - c < 4 ? p.d - c : 4);
  f64x4 sum = {0.0, 0.0, 0.0, 0.0};
  const float* at = p.partial + 2 * int64_t{chunk} * p.d + c;
  if (count == 4) {
#pragma unroll 16
    for (int k = from; k < to; ++k)
      sum += __builtin_convertvector(static_cast<f32x4>(*reinterpret_cast<const f32x4_at4*>(at + (k == 0 ? 1 : 2 * int64_t{k}) * p.d)), f64x4);
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
    double all = parts[0][2 * t + i / 4][i % 4];
#pragma unroll
    for (int s = 1; s < kCuts; ++s) all += parts[s][2 * t + i / 4][i % 4];
    out[i] = static_cast<float>(all);
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
hipError_t launch_sums(Sort& s, Sum& p, int64_t chunks, int id_type, hipStream_t stream) {
  const int64_t rows = p.accumulate ? 0 : p.vocab * p.column_blocks;    // to be cleared, in pieces of a wave
  if (p.tokens <= kFewTokens) {
    p.tasks = p.tokens * p.column_blocks;
    const unsigned few = static_cast<unsigned>(pieces_of(p.tasks + rows, 4));
    return id_type == OPT8_ID_INT32 ? queue(few_kernel<X, D, int32_t>, few, 256, stream, p)
                                    : queue(few_kernel<X, D, int64_t>, few, 256, stream, p);
  }
  const unsigned groups = static_cast<unsigned>(s.shape.groups);
  hipError_t e = id_type == OPT8_ID_INT32 ? queue(sort_kernel<int32_t>, groups, 64 * kSortWaves, stream, s)
                                          : queue(sort_kernel<int64_t>, groups, 64 * kSortWaves, stream, s);
  const int64_t sums = p.sum_groups + pieces_of(rows, 4);
  if (e == hipSuccess) e = queue(sum_kernel<X, D>, static_cast<unsigned>(sums), 256, stream, p);
  if (e == hipSuccess && chunks > 1)
    e = queue(join_kernel<D>, static_cast<unsigned>((chunks - 1) * pieces_of(p.d, 1024)), 256 * kCuts, stream, p);
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
  s.shape = sort_shape(a.vocab);
  s.order = reinterpret_cast<int*>(work + space.order);
  s.keys = reinterpret_cast<int*>(work + space.keys);
  s.starts = reinterpret_cast<int*>(work + space.starts);
  Sum p;
  p.ids = a.ids;
  p.tokens = a.tokens;
  p.order = s.order;
  p.keys = s.keys;
  p.starts = s.starts;
  p.shape = s.shape;
  p.dy = a.dy;
  p.dtable = a.dtable;
  p.partial = reinterpret_cast<float*>(work + space.partial);
  p.vocab = a.vocab;
  p.d = a.d;
  p.lddy = a.lddy;
  p.lddtable = a.lddtable;
  p.scale = a.scale;
  p.accumulate = a.accumulate != 0;
  p.stream = streams(2 * a.d * (a.tokens + (p.accumulate ? a.tokens : a.vocab)));
  p.chunk = static_cast<int>(sum_chunk(a.tokens, a.d));
  p.column_blocks = static_cast<int>(pieces_of(a.d, 512));
  const int64_t chunks = pieces_of(a.tokens, p.chunk);
  p.tasks = chunks * p.column_blocks;
  p.sum_groups = pieces_of(p.tasks, 4);
  const bool wide = a.dtable_type == OPT8_TYPE_FP32;
  if (a.type == OPT8_TYPE_BF16) return wide ? launch_sums<Bf16, float>(s, p, chunks, a.id_type, stream) : launch_sums<Bf16, Bf16>(s, p, chunks, a.id_type, stream);
  if (a.type == OPT8_TYPE_FP16) return wide ? launch_sums<Fp16, float>(s, p, chunks, a.id_type, stream) : launch_sums<Fp16, Fp16>(s, p, chunks, a.id_type, stream);
  return launch_sums<float, float>(s, p, chunks, a.id_type, stream);
}

}  // namespace opt8
