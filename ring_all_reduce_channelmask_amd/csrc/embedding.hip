// embedding.hip -- token embeddings from a table split by vocabulary over the
// ranks, and their gradient.
//
//   forward   y_k[t] = scale * E[ids[t]]                       k = every copy
//   gradient  dE[v] (+)= scale * sum over t with ids[t] = v of sum_k dy_k[t]
//
// The one-shot AllReduce of a split lookup has one term that is not zero, the
// owner's: it alone is read.  The gradient groups equal tokens, in order of
// their positions, and adds up each group in fp32: up to 1024 tokens four waves
// a quarter of it each, beyond that the chunks of the ordered list their parts,
// which are joined.  No float is added atomically, and the parts depend on the
// sizes and the ids alone, so the same inputs give the same bits.
//
// Bound by memory.  Measured (kernels, bf16): 4096 tokens of 7168, 4 copies 38 us
// (235 MB written, 6.1 TB/s; a text's frequent rows come from the caches: with
// loads that bypass them 59), 1 token 3.1 us; gradient of 65536 tokens of 2048
// (vocabulary 131072) 24 us for the order, 162 for the sums and the zeros (805
// MB: 5.0 TB/s) and 15 for the groups that chunks cut (added to 20000 rows of the
// table, not dense: 101 for the sums; in an fp32 table 307 dense, 237 added to); of
// 333 tokens of 1001 in fp32 13 us (32 MB written).
#include "op_common.h"

namespace rar {
namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxVocab = int64_t(1) << 30;
constexpr int64_t kMaxWidth = int64_t(1) << 24;
typedef float v4f_user __attribute__((ext_vector_type(4), aligned(4)));
constexpr int kRow = 512;        // 16-bit elements of a wave's piece of a row (256 of 32 bits)
// Up to kSmallTokens a group's positions are found by looking at all ids, in
// one launch (1000 tokens of 4096: 64 us; 1100 in three launches 63).  Up to
// kRankTokens the order comes from comparing all pairs (4096 tokens 9.3 us,
// 16384 27; the radix sort 22 to 24 whatever the number there).
constexpr int kSmallTokens = 1024;
constexpr int kRankTokens = 8192;

// Where the ranks' rows begin in the vocabulary; first[nranks] is its size.
struct Split {
  int32_t first[kMaxRanks + 1];
  int32_t nranks;
  __device__ __forceinline__ int rank_of(int32_t v) const {
    int r = 0;
    while (first[r + 1] <= v) ++r;
    return r;
  }
};

struct ForwardArgs {
  const void* table[kMaxRanks];
  int64_t table_stride[kMaxRanks];
  void* dst[kMaxRanks];
  int64_t dst_stride[kMaxRanks];
  const int64_t* ids;
  int64_t tokens, width, pieces;  // pieces of a row
  float scale;
  int32_t ndst;
  uint32_t block0;  // workgroups in earlier launches
  Split split;
};

// kThreads threads (64 or 256) take kVecs vectors each of one token's row.
template <class T, int kVecs, int kThreads>
__global__ void __launch_bounds__(256) embedding_kernel(ForwardArgs) {
  const ForwardArgs& args = kernel_args<ForwardArgs>();
  const int64_t item = (int64_t)(args.block0 + blockIdx.x) * (256 / kThreads) + threadIdx.x / kThreads;
  const int64_t t = item / args.pieces, piece = item - t * args.pieces;
  if (t >= args.tokens) return;
  const int64_t id = args.ids[t];
  const int64_t e0 = piece * (kThreads * kVecs * T::kVec) + threadIdx.x % kThreads * T::kVec;
  v4u v[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) v[j] = v4u{0, 0, 0, 0};
  if (id >= 0 && id < args.split.first[args.split.nranks]) {
    const int r = args.split.rank_of((int32_t)id);
    const typename T::bits* src = static_cast<const typename T::bits*>(args.table[r]) + (id - args.split.first[r]) * args.table_stride[r];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) v[j] = RowEdge<T>(e0 + j * (kThreads * T::kVec), args.width).load_shared(src);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float f[T::kVec];
      RowEdge<T>(e0 + j * (kThreads * T::kVec), args.width).fix(v[j]);
      T::widen(v[j], f);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) f[i] *= args.scale;
      v[j] = T::round(f);
    }
  }
  for (int k = 0; k < args.ndst; ++k) {
    typename T::bits* dst = static_cast<typename T::bits*>(args.dst[k]) + t * args.dst_stride[k];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int64_t e = e0 + j * (kThreads * T::kVec);
      if (e < args.width) store_part<T>(dst + e, (int)(args.width - e > T::kVec ? T::kVec : args.width - e), v[j]);
    }
  }
}

// ---- gradient ----------------------------------------------------------------

struct BackwardArgs {
  const void* grad[kMaxRanks];
  int64_t grad_stride[kMaxRanks];
  void* table[kMaxRanks];
  int64_t table_stride[kMaxRanks];
  const int64_t* ids;
  int32_t* keys[2];    // ids in order, those outside the vocabulary last as its size
  int32_t* places[2];  // their positions
  uint32_t* counts;    // of the radix sort: [blocks][kDigits]
  float* partial;      // [2 * chunks][width]: groups cut by a chunk's start, its end
  int64_t tokens, width;
  int64_t slices;      // pieces of a row, one a wave
  int64_t sum_groups;  // workgroups that sum; the others fill
  float scale;
  int32_t ngrads, accumulate, chunk, chunks, sorted;  // sorted: which of keys/places is in order
  int32_t shift, blocks, fill_rows;
  uint32_t block0;  // workgroups in earlier launches
  Split split;
};

__device__ __forceinline__ int32_t key_of(int64_t id, int32_t vocab) { return id >= 0 && id < vocab ? (int32_t)id : vocab; }

// Types of the table's gradient beside T, the payload's.
template <class T, class G>
struct TableRow {
  // The wave's piece of table row v from element e on.
  static __device__ __forceinline__ typename G::bits* at(const BackwardArgs& args, int32_t v, int64_t e) {
    const int r = args.split.rank_of(v);
    return static_cast<typename G::bits*>(args.table[r]) + (int64_t)(v - args.split.first[r]) * args.table_stride[r] + e;
  }
  // Write (or add to) T::kVec elements, n of them there.
  static __device__ __forceinline__ void put(const BackwardArgs& args, typename G::bits* p, int n, const float* sum) {
    constexpr int kParts = T::kVec / G::kVec;  // vectors of G: 1 or 2
#pragma unroll
    for (int j = 0; j < kParts; ++j) {
      const int left = n - j * G::kVec < 0 ? 0 : n - j * G::kVec > G::kVec ? G::kVec : n - j * G::kVec;
      float f[G::kVec];
#pragma unroll
      for (int i = 0; i < G::kVec; ++i) f[i] = sum[j * G::kVec + i] * args.scale;
      if (left <= 0) continue;
      if (args.accumulate) {
        float old[G::kVec];
        G::widen(load_part<G>(p + j * G::kVec, left, 0), old);
#pragma unroll
        for (int i = 0; i < G::kVec; ++i) f[i] += old[i];
      }
      store_part<G>(p + j * G::kVec, left, G::round(f));
    }
  }
};

// Add up rows begin to end - 1 of a list (place_of gives the i-th's position)
// of every gradient, in that order, this lane's elements from e on; `done`
// gets each row's end.  Loads are issued kBatch at a time, whatever the rows
// belong to.
template <class T, int kBatch, class P, class F>
__device__ __forceinline__ void add_rows(const BackwardArgs& args, int begin, int end, int64_t e, float* sum, P place_of, F done) {
  const RowEdge<T> edge(e, args.width);
  int i = begin, k = 0;
  while (i < end) {
    v4u x[kBatch];
    int at = i, copy = k;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      x[j] = v4u{0, 0, 0, 0};
      if (at < end) {
        x[j] = edge.load(static_cast<const typename T::bits*>(args.grad[copy]) + place_of(at) * args.grad_stride[copy]);
        if (++copy == args.ngrads) copy = 0, ++at;
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (i < end) {
        float f[T::kVec];
        edge.fix(x[j]);
        T::widen(x[j], f);
#pragma unroll
        for (int c = 0; c < T::kVec; ++c) sum[c] += f[c];
        if (++k == args.ngrads) {
          done(i);
          k = 0, ++i;
        }
      }
    }
  }
}

// A wave zeroes its piece of table row v.
template <class G>
__device__ __forceinline__ void zero_row(const BackwardArgs& args, int32_t v, int lane) {
  const int r = args.split.rank_of(v);
  typename G::bits* p = static_cast<typename G::bits*>(args.table[r]) + (int64_t)(v - args.split.first[r]) * args.table_stride[r];
  for (int64_t e = lane * G::kVec; e < args.width; e += 64 * G::kVec)
    store_part<G>(p + e, (int)(args.width - e > G::kVec ? G::kVec : args.width - e), v4u{0, 0, 0, 0});
}

constexpr int kFillRows = 64;  // table rows that a filling workgroup looks at, at most

// Few tokens, one launch.  A summing workgroup takes a token and a piece of
// its row: if no earlier token is the same, it lists all that are, and each
// wave adds up a run of them.  A filling workgroup zeroes those of its rows
// that no token has.
template <class T, class G>
__global__ void __launch_bounds__(256) few_tokens_kernel(BackwardArgs) {
  const BackwardArgs& args = kernel_args<BackwardArgs>();
  const uint32_t block = args.block0 + blockIdx.x;
  constexpr int kRounds = kSmallTokens / 256;
  __shared__ int32_t list[kSmallTokens];
  __shared__ int32_t counts[kRounds][4];
  __shared__ float parts[3][64 * T::kVec];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t vocab = args.split.first[args.split.nranks], tokens = (int32_t)args.tokens;
  int32_t keys[kRounds];  // of tokens threadIdx.x, 256 + threadIdx.x, ...; loaded together
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int32_t u = i * 256 + threadIdx.x;
    keys[i] = u < tokens ? key_of(args.ids[u], vocab) : vocab;
  }
  if (block >= args.sum_groups) {
    const int32_t r0 = (int32_t)(block - args.sum_groups) * args.fill_rows, r1 = std::min(vocab, r0 + args.fill_rows);
    int32_t* used = list;
    if (threadIdx.x < kFillRows) used[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      if (keys[i] >= r0 && keys[i] < r1) used[keys[i] - r0] = 1;
    __syncthreads();
    for (int i = wave; r0 + i < r1; i += 4)
      if (!used[i]) zero_row<G>(args, r0 + i, lane);
    return;
  }
  const int32_t t = (int32_t)(block / args.slices);
  const int32_t key = key_of(args.ids[t], vocab);
  if (key == vocab) return;
  uint64_t same[kRounds];
  bool earlier = false;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    same[i] = __ballot(keys[i] == key);
    earlier = earlier || (keys[i] == key && i * 256 + (int32_t)threadIdx.x < t);
    if (lane == 0) counts[i][wave] = __popcll(same[i]);
  }
  if (__syncthreads_or(earlier)) return;
  int total = 0;
#pragma unroll
  for (int i = 0; i < kRounds; ++i)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w == wave && keys[i] == key) list[total + bits_below(same[i])] = i * 256 + threadIdx.x;
      total += counts[i][w];
    }
  __syncthreads();
  const int64_t e = (block - t * args.slices) * (64 * T::kVec) + lane * T::kVec;
  const int n = (int)(args.width - e >= T::kVec ? T::kVec : args.width - e < 0 ? 0 : args.width - e);
  float sum[T::kVec];
#pragma unroll
  for (int c = 0; c < T::kVec; ++c) sum[c] = 0.0f;
  total = __builtin_amdgcn_readfirstlane(total);
  add_rows<T, 16>(args, (total * wave + 3) / 4, (total * (wave + 1) + 3) / 4, e, sum,
                 [&](int i) { return (int64_t)__builtin_amdgcn_readfirstlane(list[i]); }, [](int) {});
  if (total > 1) {  // otherwise the first wave has the only row
    if (wave > 0) {
#pragma unroll
      for (int c = 0; c < T::kVec; ++c) parts[wave - 1][c * 64 + lane] = sum[c];
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 3; ++w)
#pragma unroll
      for (int c = 0; c < T::kVec; ++c) sum[c] += parts[w][c * 64 + lane];
  }
  if (wave == 0) TableRow<T, G>::put(args, TableRow<T, G>::at(args, key, e), n, sum);
}

// The order of up to kRankTokens tokens: each one's place is the number of
// smaller keys, or equal ones before it.  A workgroup places 64 tokens, one a
// lane; its 16 waves share the keys they are compared with.
__global__ void __launch_bounds__(1024) rank_kernel(BackwardArgs) {
  const BackwardArgs& args = kernel_args<BackwardArgs>();
  __shared__ __attribute__((aligned(16))) int32_t keys[kRankTokens];
  __shared__ int32_t counts[16][64];
  const int32_t vocab = args.split.first[args.split.nranks], tokens = (int32_t)args.tokens;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t padded = (tokens + 63) & ~63;
  for (int32_t u = threadIdx.x; u < padded; u += 1024) keys[u] = u < tokens ? key_of(args.ids[u], vocab) : 0x7FFFFFFF;
  __syncthreads();
  const int32_t t0 = blockIdx.x * 64, t = t0 + lane;
  const int32_t key = keys[t];  // t < padded
  int32_t below = 0;
  // 64 keys at a time: those before the workgroup's tokens count where they
  // are equal, those behind do not
  for (int32_t u0 = wave * 64; u0 < padded; u0 += 16 * 64) {
    if (u0 == t0) {
      for (int i = 0; i < 64; ++i) {
        const int32_t other = keys[u0 + i];
        below += other < key || (other == key && i < lane);
      }
    } else {
      const int32_t bound = u0 < t0 ? key + 1 : key;
      for (int i = 0; i < 64; i += 4) {
        const v4u other = *reinterpret_cast<const v4u*>(&keys[u0 + i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) below += (int32_t)other[j] < bound;
      }
    }
  }
  counts[wave][lane] = below;
  __syncthreads();
  if (wave == 0 && t < tokens) {
    int32_t place = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) place += counts[w][lane];
    args.keys[0][place] = key;
    args.places[0][place] = t;
  }
}

// More tokens: a radix sort, 9 bits of the key a pass.  `blocks` workgroups
// each take a run of tokens; count_kernel counts their digits, place_kernel
// puts each token behind the smaller digits, the same digit of earlier runs
// and of earlier tokens of its own.
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits, kSortThreads = 1024;

__device__ __forceinline__ void run_of(const BackwardArgs& args, int64_t* begin, int64_t* end) {
  const int64_t len = (args.tokens + args.blocks - 1) / args.blocks;
  *begin = std::min<int64_t>(args.tokens, blockIdx.x * len);
  *end = std::min<int64_t>(args.tokens, *begin + len);
}
__device__ __forceinline__ int32_t sort_key(const BackwardArgs& args, int64_t t, int32_t vocab) {
  return args.shift == 0 ? key_of(args.ids[t], vocab) : args.keys[1 - args.sorted][t];
}
__global__ void __launch_bounds__(kSortThreads) count_kernel(BackwardArgs) {
  const BackwardArgs& args = kernel_args<BackwardArgs>();
  __shared__ uint32_t counts[kDigits];
  const int32_t vocab = args.split.first[args.split.nranks];
  if (threadIdx.x < kDigits) counts[threadIdx.x] = 0;
  __syncthreads();
  int64_t begin, end;
  run_of(args, &begin, &end);
#pragma unroll 4
  for (int64_t t = begin + threadIdx.x; t < end; t += kSortThreads)
    atomicAdd(&counts[(sort_key(args, t, vocab) >> args.shift) & (kDigits - 1)], 1u);
  __syncthreads();
  if (threadIdx.x < kDigits) args.counts[blockIdx.x * kDigits + threadIdx.x] = counts[threadIdx.x];
}
__global__ void __launch_bounds__(kSortThreads) place_kernel(BackwardArgs) {
  const BackwardArgs& args = kernel_args<BackwardArgs>();
  constexpr int kWaves = kSortThreads / 64, kHalves = kSortThreads / kDigits;
  __shared__ uint32_t next[kDigits], seen[kWaves][kDigits], sums[kWaves], half[kHalves][2][kDigits];
  const int32_t vocab = args.split.first[args.split.nranks];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, mine = threadIdx.x % kDigits;
  {  // digit `mine`: in the runs before this one, and in all; each half of the threads takes every other run
    uint32_t before = 0, total = 0;
#pragma unroll 16
    for (int b = threadIdx.x / kDigits; b < args.blocks; b += kHalves) {
      const uint32_t c = args.counts[b * kDigits + mine];
      before += b < (int)blockIdx.x ? c : 0;
      total += c;
    }
    half[threadIdx.x / kDigits][0][mine] = before;
    half[threadIdx.x / kDigits][1][mine] = total;
  }
  __syncthreads();
  uint32_t before = 0, total = 0, upto = 0;
  if (threadIdx.x < kDigits) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h) before += half[h][0][mine], total += half[h][1][mine];
    upto = total;
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t other = __shfl_up(upto, d);
      if (lane >= d) upto += other;
    }
    if (lane == 63) sums[wave] = upto;
  }
  __syncthreads();
  if (threadIdx.x < kDigits) {
    uint32_t start = upto - total + before;
    for (int w = 0; w < wave; ++w) start += sums[w];
    next[mine] = start;
  }
  int64_t begin, end;
  run_of(args, &begin, &end);
  for (int64_t t0 = begin; t0 < end; t0 += kSortThreads) {
    for (int i = threadIdx.x; i < kWaves * kDigits; i += kSortThreads) seen[0][i] = 0;
    __syncthreads();
    const int64_t t = t0 + threadIdx.x;
    const bool in = t < end;
    const int32_t key = in ? sort_key(args, t, vocab) : 0;
    const int32_t place = !in ? 0 : args.shift == 0 ? (int32_t)t : args.places[1 - args.sorted][t];
    const int digit = (key >> args.shift) & (kDigits - 1);
    uint64_t same = __ballot(in);
#pragma unroll
    for (int bit = 0; bit < kDigitBits; ++bit) {
      const uint64_t ones = __ballot(digit >> bit & 1);
      same &= digit >> bit & 1 ? ones : ~ones;
    }
    const int above = bits_below(same);
    if (in && above == 0) seen[wave][digit] = __popcll(same);
    __syncthreads();
    if (threadIdx.x < kDigits) {  // where each wave's tokens of the digit begin
      uint32_t at = next[mine];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const uint32_t c = seen[w][mine];
        seen[w][mine] = at;
        at += c;
      }
      next[mine] = at;
    }
    __syncthreads();
    if (in) {
      const uint32_t at = seen[wave][digit] + above;
      args.keys[args.sorted][at] = key;
      args.places[args.sorted][at] = place;
    }
    __syncthreads();
  }
}

// The first place of [0, n) whose key is at least v: a wave narrows the range
// 64 times a step.
__device__ __forceinline__ int64_t lower_bound(const int32_t* keys, int64_t n, int32_t v, int lane) {
  int64_t lo = 0, hi = n;  // the answer is in [lo, hi]
  while (hi > lo) {
    const int64_t step = (hi - lo + 63) / 64, at = lo + lane * step;
    const int below = __popcll(__ballot(at < hi && keys[at < hi ? at : lo] < v));  // a prefix of the lanes
    if (below == 0) return lo;
    lo += (below - 1) * step + 1;  // keys[lo + (below - 1) * step] < v
    hi = std::min(hi, lo - 1 + step);
  }
  return lo;
}

// A summing wave takes `chunk` (up to 64) tokens in order and a piece of the
// row.  A group within the chunk goes to its table row; what belongs to a
// group that other chunks share goes to `partial`: to 2c what continues from
// the chunk before, to 2c + 1 what begins in this one and goes on.
template <class T, class G>
__global__ void __launch_bounds__(256) sum_kernel(BackwardArgs) {
  const BackwardArgs& args = kernel_args<BackwardArgs>();
  const uint32_t block = args.block0 + blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t vocab = args.split.first[args.split.nranks];
  const int32_t* keys = args.keys[args.sorted];
  if (block >= args.sum_groups) {
    __shared__ uint32_t used[kFillRows];
    const int32_t r0 = (int32_t)(block - args.sum_groups) * args.fill_rows, r1 = std::min(vocab, r0 + args.fill_rows);
    if (threadIdx.x < kFillRows) used[threadIdx.x] = 0;
    __syncthreads();
    if (wave == 0) {
      const int64_t end = lower_bound(keys, args.tokens, r1, lane);
      for (int64_t i = lower_bound(keys, args.tokens, r0, lane) + lane; i < end; i += 64) used[keys[i] - r0] = 1;
    }
    __syncthreads();
    for (int i = wave; r0 + i < r1; i += 4)
      if (!used[i]) zero_row<G>(args, r0 + i, lane);
    return;
  }
  const int64_t item = (int64_t)block * 4 + wave;
  const int64_t c = item / args.slices;
  if (c >= args.chunks) return;
  const int64_t e = (item - c * args.slices) * (64 * T::kVec) + lane * T::kVec;
  const int n = (int)(args.width - e >= T::kVec ? T::kVec : args.width - e < 0 ? 0 : args.width - e);
  const int64_t i0 = c * args.chunk;
  const int len = (int)std::min<int64_t>(args.chunk, args.tokens - i0);
  const int32_t key = lane < len ? keys[i0 + lane] : vocab;
  const int32_t place = lane < len ? args.places[args.sorted][i0 + lane] : 0;
  const int32_t last = i0 > 0 ? keys[i0 - 1] : -1, next = i0 + len < args.tokens ? keys[i0 + len] : -1;
  // lanes that end a group, the chunk's last token among them; those outside
  // the vocabulary are behind all others
  const int32_t down = __shfl_down(key, 1);
  const int used = __popcll(__ballot(lane < len && key != vocab));
  const uint64_t ends = __ballot(lane < used && (lane == used - 1 || key != down));
  float sum[T::kVec];
#pragma unroll
  for (int i = 0; i < T::kVec; ++i) sum[i] = 0.0f;
  int begin = 0;
  add_rows<T, 8>(args, 0, used, e, sum, [&](int i) { return (int64_t)__builtin_amdgcn_readlane(place, i); },
                 [&](int i) {
                   if (!(ends >> i & 1)) return;
                   const int32_t v = __builtin_amdgcn_readlane(key, i);
                   const bool from = begin == 0 && last == v, on = i + 1 == len && next == v;
                   if (from || on) {
                     float* p = args.partial + (2 * c + !from) * args.width + e;
#pragma unroll
                     for (int j = 0; j < T::kVec / 4; ++j) store4<F32>(reinterpret_cast<uint32_t*>(p + 4 * j), n - 4 * j, sum + 4 * j);
                   } else {
                     TableRow<T, G>::put(args, TableRow<T, G>::at(args, v, e), n, sum);
                   }
#pragma unroll
                   for (int j = 0; j < T::kVec; ++j) sum[j] = 0.0f;
                   begin = i + 1;
                 });
}

// The groups cut by chunks: the workgroup of the chunk where one begins adds
// up its parts for kJoinColumns columns, each of kJoinWaves waves a run of them.
constexpr int kJoinWaves = 4, kJoinColumns = 512, kJoinVecs = kJoinColumns / 256;
template <class T, class G>
__global__ void __launch_bounds__(64 * kJoinWaves) join_kernel(BackwardArgs) {
  const BackwardArgs& args = kernel_args<BackwardArgs>();
  const uint32_t block = args.block0 + blockIdx.x;
  __shared__ float parts[kJoinWaves][kJoinColumns];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t vocab = args.split.first[args.split.nranks];
  const int32_t* keys = args.keys[args.sorted];
  const int64_t slices = (args.width + kJoinColumns - 1) / kJoinColumns;
  const int64_t c = block / slices, e = (block - c * slices) * kJoinColumns + lane * 4;
  const int64_t i0 = c * args.chunk, i1 = i0 + args.chunk;  // not the last chunk
  const int32_t v = keys[i1 - 1], first = keys[i0], before = i0 > 0 ? keys[i0 - 1] : -1;
  if (v == vocab || keys[i1] != v || (first == v && before == v)) return;
  // chunks c + 1 ... c + more hold the rest of the group
  int64_t more = 0;
  for (;; more += 64) {
    const int64_t i = (c + 1 + more + lane) * args.chunk;
    const uint64_t same = __ballot(i < args.tokens && keys[i < args.tokens ? i : 0] == v);
    if (same != ~uint64_t(0)) {
      more += __builtin_ctzll(~same);
      break;
    }
  }
  // part 0 is the chunk's own, part j that of chunk c + j
  const int64_t each = (more + kJoinWaves) / kJoinWaves, j0 = wave * each, j1 = std::min<int64_t>(more + 1, j0 + each);
  float sum[kJoinVecs * 4];
#pragma unroll
  for (int i = 0; i < kJoinVecs * 4; ++i) sum[i] = 0.0f;
  constexpr int kBatch = 8;
  for (int64_t b = j0; b < j1; b += kBatch) {
    v4f_user x[kBatch][kJoinVecs];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t j = std::min(b + i, j1 - 1);
      const float* p = args.partial + (j == 0 ? 2 * c + 1 : 2 * (c + j)) * args.width;
      // beyond the row's end there is the next one, or the slack behind the last
#pragma unroll
      for (int h = 0; h < kJoinVecs; ++h) x[i][h] = *reinterpret_cast<const v4f_user*>(p + (e + h * 256 < args.width ? e + h * 256 : 0));
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (b + i < j1)
#pragma unroll
        for (int h = 0; h < kJoinVecs; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) sum[h * 4 + k] += x[i][h][k];
  }
#pragma unroll
  for (int h = 0; h < kJoinVecs; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) parts[wave][h * 256 + lane * 4 + i] = sum[h * 4 + i];
  __syncthreads();
  for (int i = threadIdx.x; i < kJoinColumns; i += 64 * kJoinWaves) {
    const int64_t column = (block - c * slices) * kJoinColumns + i;
    if (column >= args.width) return;
    float all = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) all += parts[w][i];
    typename G::bits* p = TableRow<T, G>::at(args, v, column);
    float f = all * args.scale;
    if (args.accumulate) f += G::widen1(*p);
    *p = G::round1(f);
  }
}

// ---- host --------------------------------------------------------------------

int64_t align_up(int64_t n) { return (n + 255) & ~int64_t(255); }

// How the gradient of a call is cut, and where its workspace holds what.
struct Shape {
  int32_t chunk = 0, chunks = 0, blocks = 0, bits = 0;
  int64_t keys = 0, counts = 0, partial = 0, bytes = 0;
};
Shape shape_of(int64_t tokens, int64_t width, int64_t vocab) {
  Shape s;
  if (tokens <= kSmallTokens) return s;
  // as many waves as the device holds (8192), in chunks of 8 to 64 tokens; by
  // pieces of 512 elements, of which fp32 takes two waves each
  const int64_t slices = (width + kRow - 1) / kRow;
  s.chunk = 64;
  while (s.chunk > 8 && tokens / s.chunk * slices < 8192) s.chunk /= 2;
  s.chunks = (int32_t)((tokens + s.chunk - 1) / s.chunk);
  while ((vocab >> s.bits) != 0) ++s.bits;
  s.blocks = (int32_t)std::min<int64_t>(256, (tokens + kSortThreads - 1) / kSortThreads);
  s.keys = align_up(tokens * 4);
  s.counts = align_up((int64_t)s.blocks * kDigits * 4);
  s.partial = align_up(2 * (int64_t)s.chunks * width * 4 + 16);
  s.bytes = 4 * s.keys + s.counts + s.partial;
  return s;
}

rar_result_t check_split(const int64_t* rows, int nranks, Split* split) {
  if (nranks < 1 || nranks > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "nranks must be in [1, 64]");
  if (!rows) return set_error(RAR_INVALID_ARGUMENT, "rows is NULL");
  int64_t total = 0;
  for (int r = 0; r < nranks; ++r) {
    split->first[r] = (int32_t)total;
    if (rows[r] < 0 || rows[r] > kMaxVocab || (total += rows[r]) > kMaxVocab)
      return set_error(RAR_INVALID_ARGUMENT, "the vocabulary must have 1 to 2^30 rows, none negative");
  }
  if (total < 1) return set_error(RAR_INVALID_ARGUMENT, "the vocabulary must have 1 to 2^30 rows, none negative");
  split->first[nranks] = (int32_t)total;
  split->nranks = nranks;
  return RAR_SUCCESS;
}

rar_result_t check_sizes(int64_t tokens, int64_t width, int dtype, float scale) {
  if (rar_result_t r = check_float_dtype(dtype)) return r;
  if (tokens < 0 || tokens > kMaxTokens) return set_error(RAR_INVALID_ARGUMENT, "tokens must be in [0, 2^24]");
  if (width < 1 || width > kMaxWidth) return set_error(RAR_INVALID_ARGUMENT, "width must be in [1, 2^24]");
  if (!(scale - scale == 0.0f)) return set_error(RAR_INVALID_ARGUMENT, "scale must be finite");
  return RAR_SUCCESS;
}

template <class T>
const void* forward_kernel(int threads, int vecs) {
  if (threads == 64) return reinterpret_cast<const void*>(&embedding_kernel<T, 1, 64>);
  return vecs == 2 ? reinterpret_cast<const void*>(&embedding_kernel<T, 2, 256>) : reinterpret_cast<const void*>(&embedding_kernel<T, 1, 256>);
}

rar_result_t forward(const void* const* tables, const int64_t* rows, const int64_t* table_strides, int nranks, int64_t width, int dtype,
                     const int64_t* ids, int64_t tokens, float scale, void* const* recvbufs, const int64_t* recv_strides, int nrecv,
                     void* stream) {
  ForwardArgs a{};
  if (rar_result_t r = check_split(rows, nranks, &a.split)) return r;
  if (nrecv < 1 || nrecv > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "nrecv must be in [1, 64]");
  if (rar_result_t r = check_sizes(tokens, width, dtype, scale)) return r;
  if (tokens == 0) return RAR_SUCCESS;
  if (!tables || !recvbufs) return set_error(RAR_INVALID_ARGUMENT, "an array of buffers is NULL");
  const int64_t es = elem_size(dtype);
  std::vector<Block> reads, writes;
  reads.reserve(nranks + 1);
  writes.reserve(nrecv);
  for (int r = 0; r < nranks; ++r) {
    if (rar_result_t e = set_stride(a.table_stride[r], table_strides, r, width, rows[r], "table stride")) return e;
    if (rows[r] == 0) continue;
    if (rar_result_t e = check_pointer(tables[r], es, "table", r)) return e;
    a.table[r] = tables[r];
    reads.push_back({tables[r], rows[r], width * es, a.table_stride[r] * es, "a table"});
  }
  if (rar_result_t r = check_pointer(ids, 8, "ids")) return r;
  reads.push_back({ids, 1, tokens * 8, tokens * 8, "ids"});
  for (int k = 0; k < nrecv; ++k) {
    if (rar_result_t e = set_stride(a.dst_stride[k], recv_strides, k, width, tokens, "output stride")) return e;
    if (rar_result_t e = check_pointer(recvbufs[k], es, "output", k)) return e;
    a.dst[k] = recvbufs[k];
    writes.push_back({recvbufs[k], tokens, width * es, a.dst_stride[k] * es, "output"});
  }
  if (rar_result_t r = check_blocks(reads, writes)) return r;
  a.ids = ids;
  a.width = width;
  a.scale = scale;
  a.ndst = nrecv;
  const int vec = dtype == kFloat32 ? F32::kVec : BF16::kVec;
  // a wave a row where that is enough for it, else a workgroup a piece
  const int threads = width <= 64 * vec ? 64 : 256;
  const int vecs = threads == 256 && tokens * ((width + 256 * vec - 1) / (256 * vec)) > 2048 ? 2 : 1;
  a.tokens = tokens;
  a.pieces = (width + threads * vec * vecs - 1) / (threads * vec * vecs);
  const int64_t groups = (tokens * a.pieces + 256 / threads - 1) / (256 / threads);
  if (groups > kMaxGroups) return set_error(RAR_INVALID_ARGUMENT, "tokens * width is too large");
  const void* fn = dtype == kFloat32 ? forward_kernel<F32>(threads, vecs) : forward_kernel<BF16>(threads, vecs);
  return launch_groups(fn, groups, 256, &a, &a.block0, stream);
}

template <class T, class G>
rar_result_t launch_sums(BackwardArgs& a, int64_t fill_groups, int64_t joins, void* stream) {
  if (joins == 0) return launch_groups(reinterpret_cast<const void*>(&few_tokens_kernel<T, G>), a.sum_groups + fill_groups, 256, &a, &a.block0, stream);
  if (rar_result_t r = launch_groups(reinterpret_cast<const void*>(&sum_kernel<T, G>), a.sum_groups + fill_groups, 256, &a, &a.block0, stream)) return r;
  return launch_groups(reinterpret_cast<const void*>(&join_kernel<T, G>), joins, 64 * kJoinWaves, &a, &a.block0, stream);
}

rar_result_t backward(const void* const* grads, const int64_t* grad_strides, int ngrads, int64_t tokens, int64_t width, int dtype,
                      const int64_t* ids, float scale, void* const* dtables, const int64_t* rows, const int64_t* dtable_strides, int nranks,
                      int table_dtype, int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  BackwardArgs a{};
  if (rar_result_t r = check_split(rows, nranks, &a.split)) return r;
  if (ngrads < 1 || ngrads > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "ngrads must be in [1, 64]");
  if (rar_result_t r = check_sizes(tokens, width, dtype, scale)) return r;
  if (table_dtype != dtype && table_dtype != RAR_FLOAT32) return set_error(RAR_INVALID_ARGUMENT, "the table's gradient must have the gradients' dtype or float32");
  if (accumulate != 0 && accumulate != 1) return set_error(RAR_INVALID_ARGUMENT, "accumulate must be 0 or 1");
  if (tokens == 0 && accumulate) return RAR_SUCCESS;
  if (!dtables || (tokens > 0 && !grads)) return set_error(RAR_INVALID_ARGUMENT, "an array of buffers is NULL");
  const int64_t es = elem_size(dtype), ts = elem_size(table_dtype);
  std::vector<Block> reads, writes;
  reads.reserve(ngrads + 1);
  writes.reserve(nranks + 1);
  if (tokens > 0) {
    for (int k = 0; k < ngrads; ++k) {
      if (rar_result_t e = set_stride(a.grad_stride[k], grad_strides, k, width, tokens, "gradient stride")) return e;
      if (rar_result_t e = check_pointer(grads[k], es, "gradient", k)) return e;
      a.grad[k] = grads[k];
      reads.push_back({grads[k], tokens, width * es, a.grad_stride[k] * es, "a gradient"});
    }
    if (rar_result_t r = check_pointer(ids, 8, "ids")) return r;
    reads.push_back({ids, 1, tokens * 8, tokens * 8, "ids"});
  }
  for (int r = 0; r < nranks; ++r) {
    if (rar_result_t e = set_stride(a.table_stride[r], dtable_strides, r, width, rows[r], "table stride")) return e;
    if (rows[r] == 0) continue;
    if (rar_result_t e = check_pointer(dtables[r], ts, "table gradient", r)) return e;
    a.table[r] = dtables[r];
    writes.push_back({dtables[r], rows[r], width * ts, a.table_stride[r] * ts, "table gradient"});
  }
  const int64_t vocab = a.split.first[nranks];
  const Shape s = shape_of(tokens, width, vocab);
  if (s.bytes) {
    if (rar_result_t r = check_pointer(workspace, 1, "workspace")) return r;
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return set_error(RAR_INVALID_ARGUMENT, "workspace is not aligned to 16 bytes");
    if (workspace_bytes < (size_t)s.bytes) return set_error(RAR_INVALID_ARGUMENT, "workspace is too small");
    writes.push_back({workspace, 1, s.bytes, s.bytes, "workspace"});
  }
  if (rar_result_t r = check_blocks(reads, writes)) return r;
  a.ids = ids;
  a.tokens = tokens;
  a.width = width;
  a.scale = scale;
  a.ngrads = ngrads;
  a.accumulate = accumulate;
  a.chunk = s.chunk;
  a.chunks = s.chunks;
  a.blocks = s.blocks;
  const int64_t piece = 64 * (dtype == kFloat32 ? F32::kVec : BF16::kVec);
  a.slices = (width + piece - 1) / piece;
  a.sum_groups = s.bytes ? (s.chunks * a.slices + 3) / 4 : tokens * a.slices;
  // the groups that two chunks share; 0 where there are no chunks
  const int64_t joins = s.bytes ? (int64_t)(s.chunks - 1) * ((width + kJoinColumns - 1) / kJoinColumns) : 0;
  // enough workgroups for all CUs where the vocabulary is small
  a.fill_rows = (int32_t)std::max<int64_t>(4, std::min<int64_t>(kFillRows, vocab / 2048));
  const int64_t fill = accumulate ? 0 : (vocab + a.fill_rows - 1) / a.fill_rows;
  if (std::max(a.sum_groups + fill, joins) > kMaxGroups) return set_error(RAR_INVALID_ARGUMENT, "tokens * width is too large");
  if (s.bytes) {
    char* p = static_cast<char*>(workspace);
    for (int i = 0; i < 2; ++i) {
      a.keys[i] = reinterpret_cast<int32_t*>(p + i * s.keys);
      a.places[i] = reinterpret_cast<int32_t*>(p + (2 + i) * s.keys);
    }
    a.counts = reinterpret_cast<uint32_t*>(p + 4 * s.keys);
    a.partial = reinterpret_cast<float*>(p + 4 * s.keys + s.counts);
    if (tokens <= kRankTokens) {
      if (rar_result_t r = launch_kernel(reinterpret_cast<const void*>(&rank_kernel), dim3((unsigned)((tokens + 63) / 64)), dim3(1024), &a, stream)) return r;
    } else {
      for (a.shift = 0; a.shift < s.bits; a.shift += kDigitBits) {
        a.sorted = (a.shift / kDigitBits) & 1;
        if (rar_result_t r = launch_kernel(reinterpret_cast<const void*>(&count_kernel), dim3(s.blocks), dim3(kSortThreads), &a, stream)) return r;
        if (rar_result_t r = launch_kernel(reinterpret_cast<const void*>(&place_kernel), dim3(s.blocks), dim3(kSortThreads), &a, stream)) return r;
      }
    }
  }
  if (dtype == kFloat32) return launch_sums<F32, F32>(a, fill, joins, stream);
  return table_dtype == kFloat32 ? launch_sums<BF16, F32>(a, fill, joins, stream) : launch_sums<BF16, BF16>(a, fill, joins, stream);
}

}  // namespace
}  // namespace rar

extern "C" {

rar_result_t rar_embedding_allreduce(const void* const* tables, const int64_t* rows, const int64_t* table_strides, int nranks,
                                     int64_t width, rar_dtype_t dtype, const int64_t* ids, int64_t tokens, float scale,
                                     void* const* recvbufs, const int64_t* recv_strides, int nrecv, void* stream) {
  return rar::guarded([&] {
    return rar::forward(tables, rows, table_strides, nranks, width, dtype, ids, tokens, scale, recvbufs, recv_strides, nrecv, stream);
  });
}

rar_result_t rar_embedding_allreduce_backward(const void* const* grads, const int64_t* grad_strides, int ngrads, int64_t tokens,
                                              int64_t width, rar_dtype_t dtype, const int64_t* ids, float scale,
                                              void* const* dtables, const int64_t* rows, const int64_t* dtable_strides,
                                              int nranks, rar_dtype_t table_dtype, int accumulate, void* workspace,
                                              size_t workspace_bytes, void* stream) {
  return rar::guarded([&] {
    return rar::backward(grads, grad_strides, ngrads, tokens, width, dtype, ids, scale, dtables, rows, dtable_strides, nranks, table_dtype,
                         accumulate, workspace, workspace_bytes, stream);
  });
}

rar_result_t rar_embedding_workspace(const int64_t* rows, int nranks, int64_t tokens, int64_t width, rar_dtype_t dtype, size_t* bytes) {
  return rar::guarded([&]() -> rar_result_t {
    if (!bytes) return rar::set_error(RAR_INVALID_ARGUMENT, "bytes is NULL");
    rar::Split split{};
    if (rar_result_t r = rar::check_split(rows, nranks, &split)) return r;
    if (rar_result_t r = rar::check_sizes(tokens, width, dtype, 1.0f)) return r;
    *bytes = (size_t)rar::shape_of(tokens, width, split.first[nranks]).bytes;
    return RAR_SUCCESS;
  });
}

}  // extern "C"
