// logprobs.hip -- log probabilities of given tokens over a vocabulary split
// over N virtual ranks, with the entropy and the most probable tokens, and
// the gradient of both.
//
//   z = scale * x,  lse = log sum_j e^{z_j},  logprob = z_id - lse,
//   entropy = lse - sum_j p_j z_j,  p_j = e^{z_j - lse}
//   dx_j = scale * (g [j == id] + p_j (l - g - h (log p_j + entropy)))
// for the gradients g, h, l of logprob, entropy and lse.  A z that rounds to
// -inf is a masked token's, in every output and in the gradient.
//
// Forward: one pass over the logits.  With m a running maximum (in units of
// log 2: M = m * scale * log2 e) and d_j = x_j * scale * log2 e - M, a thread
// keeps s = sum 2^{d_j} and u = sum 2^{d_j} d_j, and rescales both by
// 2^{M - M'} (u also by the shift) when its maximum grows; two such triples
// join the same way.  Then lse = ln 2 (M + log2 s) and entropy = ln 2
// (log2 s - u / s).  All of it is fp32; exp2 and log2 are the vector unit's
// own, which err by one unit in the last place.
//
// The logits are cut into tiles that do not cross ranks, one for a wave at a
// time; a workgroup takes a run of consecutive tiles of one row.  Where there
// are few rows a row is split over several workgroups, which leave (M, s, u)
// and their best tokens in the workspace for a second kernel to join.
//
// Bound: in bf16 the vector units and memory alike.  A logit costs 5.5 plain
// operations and an exp2 at a quarter of their rate, 5.5 * 4 + 16 = 38 cycles
// for a wave's 64: 8.3 TB/s on all 1024 units at 2.4 GHz.  Measured (kernel):
// 4096 rows of 131072 bf16 without alternatives 171 us = 6.3 TB/s, 2048 rows
// of fp32 163 us = 6.6; 104 masked rows of 131075 with 5 alternatives 17.7 us
// (fp32 20.6) and 5 us for the join; 1 row of 32003 with 20 alternatives 10.0
// us, of which the alternatives are 4 us (one threshold, one list, one sort of
// about 25 keys).  The gradient is bound by memory: 4096 rows of 131072 bf16
// 344 us = 6.2 TB/s; 333 rows of 32003 fp32 with an entropy gradient 18.4 us =
// 4.6 TB/s.
#include "op_common.h"

#include <cmath>
#include <limits>

namespace rar {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWaveSize;
constexpr int kMaxWgWaves = 16;
constexpr int kVecsPerTile = 4;  // 16-byte vectors of a tile per thread
constexpr int kBackVecs = 2;     // the same, of the gradient's tile (4096 x 131072 bf16: 1 352 us, 2 338, 4 364, 8 369)
constexpr int kMaxTop = 32;
constexpr int kCandidates = 1024;  // best-token candidates a workgroup holds
constexpr int kMaxSplits = 256;
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;  // 256 threads each: a grid holds less than 2^32
constexpr int64_t kMaxRows = int64_t(1) << 23;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct Shards {
  const void* ptr[kMaxRanks];
  int64_t stride[kMaxRanks];       // elements between rows
  int32_t first[kMaxRanks + 1];    // first vocabulary id of each rank; the last entry is the vocabulary
  int32_t tile0[kMaxRanks + 1];    // first tile of each rank
  int32_t nranks;
};
struct LogprobsArgs {
  Shards x;
  int32_t splits, ntop;
  float scale, scale2;             // scale, scale * log2 e
  float least;                     // the least logit x with scale * x above -inf
  const int64_t* ids;
  float *logprob, *entropy, *lse;
  int32_t* top_ids;
  float* top_logprobs;
  v4f* parts;                      // [rows][splits] M, s, u
  uint64_t* keys;                  // [rows][splits][ntop]
};

// Forward: a wave's tile; gradient: a workgroup's.
template <class T>
constexpr int wave_tile() { return kWaveSize * kVecsPerTile * T::kVec; }
template <class T>
constexpr int block_tile() { return kThreads * kBackVecs * T::kVec; }

// A tile's vectors of one thread, those of kStride threads side by side; `left`
// columns are there, the rest is -inf.
template <class T, int kStride, int kVecs>
__device__ __forceinline__ void load_vecs(v4u* raw, const typename T::bits* src, int left, int thread, bool full) {
  if (full) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) raw[v] = load_nt(src + (v * kStride + thread) * T::kVec);
  } else {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int c = (v * kStride + thread) * T::kVec;
      raw[v] = load_part<T>(src + c, left - c, T::kNegInf);
    }
  }
}

// The rank that holds tile t (or id v, from `first`).  Uniform: scalar code.
__device__ __forceinline__ int rank_of(const int32_t* starts, int nranks, int at) {
  int r = 0;
  while (r + 1 < nranks && starts[r + 1] <= at) ++r;
  return r;
}

// A token's rank among alternatives: a larger logit first, then a lower id,
// as one whole number.  -0 and 0 are equal.
__device__ __forceinline__ uint64_t key_of(float x, int id) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t up = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (uint64_t)up << 32 | (0xFFFFFFFFu - (uint32_t)id);
}
__device__ __forceinline__ float key_logit(uint64_t key) {
  const uint32_t up = (uint32_t)(key >> 32);
  return __uint_as_float(up & 0x80000000u ? up & 0x7FFFFFFFu : ~up);
}
__device__ __forceinline__ int key_id(uint64_t key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }
// The least logit above that of `key`: what a later, higher id has to reach.
__device__ __forceinline__ float above(uint64_t key) {
  const uint64_t next = ((key >> 32) + 1) << 32;
  return key_logit(next);
}

struct Stat {
  float m, s, u;  // M in units of log 2 (-inf: nothing seen), and the sums
};
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_(float x) { return __builtin_amdgcn_logf(x); }

// Move a triple to a maximum that is no lower than its own.
__device__ __forceinline__ void shift_to(Stat& a, float m) {
  if (a.m == m) return;
  const float d = fmaxf(a.m - m, -200.0f);  // 2^-200 is 0 in fp32
  const float f = exp2_(d);
  // A triple that no longer counts is dropped, but for its NaN: far out, where
  // M's rounding exceeds the range of 2^d, its sums may be infinite.
  a.u = f > 0.0f ? f * (a.u + a.s * d) : 0.0f;
  a.s = f > 0.0f || a.s != a.s ? f * a.s : 0.0f;
  a.m = m;
}

// Reductions over a wave with lane shifts inside the vector unit (shifts by 1,
// 2, 4, 8 within a row of 16 lanes, then row 15 -> next row, rows 0-1 -> rows
// 2-3): lane 63 ends with the whole, which every lane gets.  `none` is what
// lanes without a source take.
template <class Op>
__device__ __forceinline__ float wave_reduce(float v, float none, Op op) {
#define RAR_STEP(ctrl, rows)                                                                                  \
  v = op(v, __uint_as_float(__builtin_amdgcn_update_dpp((int)__float_as_uint(none), (int)__float_as_uint(v), ctrl, rows, 0xF, false)))
  RAR_STEP(0x111, 0xF);
  RAR_STEP(0x112, 0xF);
  RAR_STEP(0x114, 0xF);
  RAR_STEP(0x118, 0xF);
  RAR_STEP(0x142, 0xA);
  RAR_STEP(0x143, 0xC);
#undef RAR_STEP
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_reduce(v, 0.0f, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ Stat wave_join(Stat a) {
  shift_to(a, wave_max(a.m));
  return Stat{a.m, wave_sum(a.s), wave_sum(a.u)};
}
// The join of `n` <= 64 triples in LDS, in every wave.
__device__ __forceinline__ Stat join_all(const Stat* stats, int n) {
  const int lane = threadIdx.x & 63;
  return wave_join(lane < n ? stats[lane] : Stat{-INFINITY, 0.0f, 0.0f});
}

// Candidates for the most probable tokens, in LDS.
struct Top {
  uint64_t key[kCandidates];
  uint64_t best[kMaxTop];
  uint32_t count[3];  // appended in round t: count[t % 3]
  float group_most[kWaveSize];
  uint64_t wave_best[kMaxWgWaves];
};

// Keep the `k` largest of the n <= kCandidates keys (all different but for
// zeros), sorted, in `best`, unused places zero.  Every thread of the
// workgroup calls it.
__device__ __forceinline__ void select_top(Top& top, int n, int k) {
  const int threads = blockDim.x;
  if ((int)threadIdx.x < k) top.best[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += threads) {
    const uint64_t mine = top.key[i];
    int above_me = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) above_me += top.key[j] > mine;
    if (above_me < k) top.best[above_me] = mine;
  }
  __syncthreads();
}

__device__ __forceinline__ uint64_t wave_max_key(uint64_t a) {
#pragma unroll
  for (int d = 1; d < kWaveSize; d <<= 1) {
    const uint64_t b = __shfl_xor((unsigned long long)a, d);
    a = a > b ? a : b;
  }
  return a;
}

// A bound that at least k of the wave's 64 values reach, to the upper 16 bits
// of the k-th largest: bit by bit from the top.  NaN where there is none.
__device__ __forceinline__ float wave_kth(float v, int k) {
  const uint32_t mine = v == v ? (uint32_t)(key_of(v, 0) >> 48) : 0u;
  uint32_t bound = 0;
#pragma unroll
  for (int bit = 15; bit >= 0; --bit) {
    const uint32_t t = bound | 1u << bit;
    if (__popcll(__ballot(mine >= t)) >= k) bound = t;
  }
  return key_logit((uint64_t)bound << 48);
}

// A row whose largest logit is so far out that d_j = fma(x_j, scale2, -M) says
// nothing (M's rounding alone passes kFar * 2^-24 = 16, or M overflows), as one
// whose tokens are all masked by the type's lowest value: the triple again,
// with z rounded before M is taken off, and M and d in units of 1.  `seen` is
// the row's triple; one without any finite z keeps M = -inf.  Every thread of
// the workgroup calls it.
constexpr float kFar = 268435456.0f;  // 2^28
template <class T>
__device__ __forceinline__ Stat rescan(const Shards& x, int64_t row, float scale, Stat seen, Stat* wave_stat) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, threads = blockDim.x, waves = threads / kWaveSize;
  float m = -INFINITY;
  for (int r = 0; r < x.nranks; ++r) {
    const typename T::bits* src = static_cast<const typename T::bits*>(x.ptr[r]) + row * x.stride[r];
    for (int c = threadIdx.x; c < x.first[r + 1] - x.first[r]; c += threads) m = fmaxf(m, T::widen1(src[c]) * scale);
  }
  m = wave_max(m);
  __syncthreads();
  if (lane == 0) wave_stat[wave].m = m;
  __syncthreads();
  m = wave_max(lane < waves ? wave_stat[lane].m : -INFINITY);
  if (m == -INFINITY) return Stat{m, seen.s, 0.0f};
  float s = 0.0f, u = 0.0f;
  for (int r = 0; r < x.nranks; ++r) {
    const typename T::bits* src = static_cast<const typename T::bits*>(x.ptr[r]) + row * x.stride[r];
    for (int c = threadIdx.x; c < x.first[r + 1] - x.first[r]; c += threads) {
      const float d = T::widen1(src[c]) * scale - m;
      const float e = exp2_(d * kLog2e);
      s += e;
      u = __builtin_fmaf(e, fmaxf(d, -200.0f), u);
    }
  }
  s = wave_sum(s);
  u = wave_sum(u);
  __syncthreads();
  if (lane == 0) wave_stat[wave] = Stat{m, s, u};
  __syncthreads();
  return Stat{m, wave_sum(lane < waves ? wave_stat[lane].s : 0.0f), wave_sum(lane < waves ? wave_stat[lane].u : 0.0f)};
}

// Results of a row from its joined triple and sorted best keys.  Every thread
// of the workgroup calls it.
template <class T>
__device__ __forceinline__ void write_row(const LogprobsArgs& a, int64_t row, Stat t, const uint64_t* best,
                                          Stat* wave_stat) {
  const bool far = !(fabsf(t.m) <= kFar);
  if (far) t = rescan<T>(a.x, row, a.scale, t, wave_stat);
  const float unit = far ? 1.0f : kLn2;
  auto logprob_of = [&](float x, float logs) {
    if (far || fabsf(x * a.scale) > kFar) return (x * a.scale - unit * t.m) - logs;
    return kLn2 * __builtin_fmaf(x, a.scale2, -t.m) - logs;
  };
  const bool empty = t.m == -INFINITY && t.s == 0.0f;  // nothing but masked tokens
  const float logs = kLn2 * log2_(t.s);
  const float lse = empty ? -INFINITY : unit * t.m + logs;
  if (threadIdx.x == 0) {
    if (a.lse) a.lse[row] = lse;
    if (a.entropy) a.entropy[row] = empty ? 0.0f : logs - unit * t.u / t.s;
    if (a.logprob) {
      const int64_t id = a.ids[row];
      float lp = 0.0f;  // no token given
      if (id >= 0 && id < a.x.first[a.x.nranks]) {
        const int r = rank_of(a.x.first, a.x.nranks, (int)id);
        const float z = T::widen1(static_cast<const typename T::bits*>(a.x.ptr[r])[row * a.x.stride[r] + (id - a.x.first[r])]);
        lp = empty ? -INFINITY : logprob_of(z, logs);
      }
      a.logprob[row] = lp;
    }
  }
  if ((int)threadIdx.x < a.ntop) {
    const uint64_t key = best[threadIdx.x];
    a.top_ids[row * a.ntop + threadIdx.x] = key ? key_id(key) : -1;
    a.top_logprobs[row * a.ntop + threadIdx.x] = key ? logprob_of(key_logit(key), logs) : -INFINITY;
  }
}

template <class T, bool kTop, int kWgWaves>
__global__ void __launch_bounds__(kWgWaves * kWaveSize) logprobs_kernel(LogprobsArgs) {
  const LogprobsArgs& args = kernel_args<LogprobsArgs>();
  constexpr int kElems = kVecsPerTile * T::kVec;  // a thread's of one tile
  constexpr int kTile = wave_tile<T>();
  __shared__ Stat wave_stat[kWgWaves];
  __shared__ std::conditional_t<kTop, Top, int> top_lds;
  const int64_t row = blockIdx.x / (uint32_t)args.splits;
  const int split = (int)(blockIdx.x % (uint32_t)args.splits);
  const int tiles = args.x.tile0[args.x.nranks];
  const int t0 = (int)((int64_t)tiles * split / args.splits), t1 = (int)((int64_t)tiles * (split + 1) / args.splits);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  Stat st{-INFINITY, 0.0f, 0.0f};
  bool masked = false;  // -inf has been met
  float cut = args.least;  // a candidate's least logit
  int held = 0;         // candidates in LDS
  bool sorted = false;  // the best of them are in top.best
  if constexpr (kTop) {
    if (threadIdx.x < 3) top_lds.count[threadIdx.x] = 0;
    __syncthreads();
  }
  // element i of this thread: column col0 + column(i)
  auto column = [&](int i) { return (i / T::kVec * kWaveSize + lane) * T::kVec + i % T::kVec; };
  int round = 0;
  for (int base = t0; base < t1; base += kWgWaves, ++round) {
    const int t = base + wave;
    const bool live = t < t1;
    const int r = rank_of(args.x.tile0, args.x.nranks, live ? t : t0);
    const int col0 = (t - args.x.tile0[r]) * kTile, width = args.x.first[r + 1] - args.x.first[r];
    const typename T::bits* src = static_cast<const typename T::bits*>(args.x.ptr[r]) + row * args.x.stride[r];
    v4u raw[kVecsPerTile];
    float most = -INFINITY, vec_most[kVecsPerTile];
    if (live) {
      const bool full = col0 + kTile <= width;
      load_vecs<T, kWaveSize, kVecsPerTile>(raw, src + col0, width - col0, lane, full);
      float x[kElems];
#pragma unroll
      for (int v = 0; v < kVecsPerTile; ++v) T::widen(raw[v], x + v * T::kVec);
#pragma unroll
      for (int v = 0; v < kVecsPerTile; ++v) {
        vec_most[v] = x[v * T::kVec];
#pragma unroll
        for (int i = 1; i < T::kVec; ++i) vec_most[v] = fmaxf(vec_most[v], x[v * T::kVec + i]);
        most = fmaxf(most, vec_most[v]);
      }
      shift_to(st, fmaxf(st.m, most * args.scale2));
      const float from = st.m == -INFINITY ? 0.0f : st.m;
      // A masked token adds e * d = 0 * -inf to u: from the first one on, d is
      // bounded for u, which costs one operation of seven for each logit.
      masked = masked || !full;
      if (!masked) {
        float s = st.s, u = st.u;
#pragma unroll
        for (int i = 0; i < kElems; ++i) {
          const float d = __builtin_fmaf(x[i], args.scale2, -from);
          const float e = exp2_(d);
          s += e;
          u = __builtin_fmaf(e, d, u);
        }
        masked = __any(u != u);
        if (!masked) st = Stat{st.m, s, u};
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < kElems; ++i) {
          const float d = __builtin_fmaf(x[i], args.scale2, -from);
          const float e = exp2_(d);
          st.s += e;
          st.u = __builtin_fmaf(e, fmaxf(d, -200.0f), st.u);
        }
      }
    }
    if constexpr (kTop) {
      Top& top = top_lds;
      if (round == 0) {
        // The k-th largest of 64 groups' maxima over the workgroup: k tokens at
        // least reach it, and seldom many more.
        const float group = group_reduce<kWgWaves>(most, [](float a, float b) { return fmaxf(a, b); });
        if (lane % kWgWaves == 0) top.group_most[wave * (kWaveSize / kWgWaves) + lane / kWgWaves] = group;
        __syncthreads();
        cut = fmaxf(cut, wave_kth(top.group_most[lane], args.ntop));
      }
      uint32_t* count = &top.count[round % 3];
      if (live && __any(most >= cut)) {
        // one reservation for the wave; few of its elements are candidates
        int mine = 0;
#pragma unroll
        for (int v = 0; v < kVecsPerTile; ++v) {
          if (!__any(vec_most[v] >= cut)) continue;
          float x[T::kVec];
          T::widen(raw[v], x);
#pragma unroll
          for (int i = 0; i < T::kVec; ++i) mine += __popcll(__ballot(x[i] >= cut));
        }
        int at = 0;
        if (lane == 0) at = (int)atomicAdd(count, (uint32_t)mine);
        at = held + __builtin_amdgcn_readfirstlane(at);
#pragma unroll
        for (int v = 0; v < kVecsPerTile; ++v) {
          if (!__any(vec_most[v] >= cut)) continue;
          float x[T::kVec];
          T::widen(raw[v], x);
#pragma unroll
          for (int i = 0; i < T::kVec; ++i) {
            const uint64_t takers = __ballot(x[i] >= cut);
            if (takers) {
              const int to = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(takers >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)takers, 0));
              if (x[i] >= cut && to < kCandidates) top.key[to] = key_of(x[i], args.x.first[r] + col0 + column(v * T::kVec + i));
              at += __popcll(takers);
            }
          }
        }
      }
      // the next round's counter: last read two rounds ago, before the last barrier
      if (threadIdx.x == 0) top.count[(round + 1) % 3] = 0;
      __syncthreads();
      int n = held + (int)*count;
      const bool over = n > kCandidates;
      sorted = sorted && n == held;
      if (over) {
        // More equal logits than the list holds: the best of what it held
        // before this round, and the round's best one by one.
        select_top(top, held, args.ntop);
        if ((int)threadIdx.x < args.ntop) top.key[threadIdx.x] = top.best[threadIdx.x];
        uint64_t last = ~0ull;
        for (int k = 0; k < args.ntop; ++k) {
          uint64_t mine = 0;
#pragma unroll 1
          for (int i = 0; i < kElems && live; ++i) {
            const int c = col0 + column(i);
            if (c >= width) continue;
            const float f = T::widen1(src[c]);
            const uint64_t key = key_of(f, args.x.first[r] + c);
            if (f >= cut && key < last && key > mine) mine = key;
          }
          mine = wave_max_key(mine);
          if (lane == 0) top.wave_best[wave] = mine;
          __syncthreads();
          last = wave_max_key(lane < kWgWaves ? top.wave_best[lane] : 0);
          if (threadIdx.x == 0) top.key[args.ntop + k] = last;
          __syncthreads();
        }
        n = 2 * args.ntop;  // unused places are zero: below every candidate
      }
      // Sorting often keeps the bound close (4096 rows of 131072, 20
      // alternatives: when 512 are held 272 us, from 16 beyond k on 218).
      if (over || n > args.ntop + 16 || (round == 0 && n > args.ntop)) {
        select_top(top, n, args.ntop);
        const uint64_t kth = top.best[args.ntop - 1];
        n = args.ntop;
        // a later round's ids are higher: an equal logit no longer counts
        if (kth) cut = above(kth);
        else
          for (n = 0; top.best[n];) ++n;
        if ((int)threadIdx.x < n) top.key[threadIdx.x] = top.best[threadIdx.x];
        sorted = true;
        __syncthreads();
      }
      held = n;
    }
  }
  st = wave_join(st);
  if (lane == 0) wave_stat[wave] = st;
  __syncthreads();
  st = join_all(wave_stat, kWgWaves);
  const uint64_t* best = nullptr;
  if constexpr (kTop) {
    if (!sorted) select_top(top_lds, held, args.ntop);
    best = top_lds.best;
  }
  if (args.splits == 1) {
    write_row<T>(args, row, st, best, wave_stat);
    return;
  }
  if (threadIdx.x == 0) args.parts[blockIdx.x] = v4f{st.m, st.s, st.u, 0.0f};
  if constexpr (kTop) {
    if ((int)threadIdx.x < args.ntop) args.keys[(int64_t)blockIdx.x * args.ntop + threadIdx.x] = best[threadIdx.x];
  }
}

// Join a row's parts: one workgroup a row.
template <class T>
__global__ void __launch_bounds__(kThreads) logprobs_join_kernel(LogprobsArgs) {
  const LogprobsArgs& args = kernel_args<LogprobsArgs>();
  __shared__ Stat wave_stat[kWaves];
  __shared__ Top top;
  const int64_t row = blockIdx.x;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  Stat st{-INFINITY, 0.0f, 0.0f};
  if ((int)threadIdx.x < args.splits) {
    const v4f p = args.parts[row * args.splits + threadIdx.x];
    st = Stat{p[0], p[1], p[2]};
  }
  st = wave_join(st);
  if (lane == 0) wave_stat[wave] = st;
  if (args.ntop) {
    // Only keys that reach the largest of the parts' k-th keys can be among the best k.
    const uint64_t* keys = args.keys + row * args.splits * args.ntop;
    uint64_t least = 0;
    if ((int)threadIdx.x < args.splits) least = keys[threadIdx.x * args.ntop + args.ntop - 1];
    least = wave_max_key(least);
    if (lane == 0) top.wave_best[wave] = least;
    if (threadIdx.x == 0) top.count[0] = 0;
    __syncthreads();
    least = wave_max_key(lane < kWaves ? top.wave_best[lane] : 0);
    for (int i = threadIdx.x; i < args.splits * args.ntop; i += kThreads) {
      const uint64_t key = keys[i];
      if (key && key >= least) top.key[atomicAdd(&top.count[0], 1u)] = key;
    }
    __syncthreads();
    select_top(top, (int)top.count[0], args.ntop);
  } else {
    __syncthreads();
  }
  write_row<T>(args, row, join_all(wave_stat, kWaves), top.best, wave_stat);
}

struct LogprobsBackwardArgs {
  Shards x;
  void* grad[kMaxRanks];
  int64_t grad_stride[kMaxRanks];
  int64_t row0;
  float scale;
  const int64_t* ids;
  const float *lse, *entropy, *grad_logprob, *grad_entropy, *grad_lse;
};

// One tile of one row a workgroup.  With w = l - g - h * entropy the gradient
// is scale * (p_j (w - h log p_j) + g [j == id]).  Bound by memory: every
// logit read and every gradient written once.
template <class T, bool kEntropy>
__global__ void __launch_bounds__(kThreads) logprobs_backward_kernel(LogprobsBackwardArgs) {
  const LogprobsBackwardArgs& args = kernel_args<LogprobsBackwardArgs>();
  constexpr int kTile = block_tile<T>();
  const uint32_t tiles = (uint32_t)args.x.tile0[args.x.nranks];
  const int64_t row = args.row0 + blockIdx.x / tiles;
  const int t = (int)(blockIdx.x % tiles);
  const int r = rank_of(args.x.tile0, args.x.nranks, t);
  const int col0 = (t - args.x.tile0[r]) * kTile;
  const int width = args.x.first[r + 1] - args.x.first[r];
  const typename T::bits* src = static_cast<const typename T::bits*>(args.x.ptr[r]) + row * args.x.stride[r];
  typename T::bits* dst = static_cast<typename T::bits*>(args.grad[r]) + row * args.grad_stride[r];
  v4u raw[kBackVecs];
  load_vecs<T, kThreads, kBackVecs>(raw, src + col0, width - col0, threadIdx.x, col0 + kTile <= width);
  const float lse = args.lse[row];
  const bool empty = lse == -INFINITY;
  const int64_t id = args.ids[row];
  const bool given = id >= 0 && id < args.x.first[args.x.nranks] && !empty;
  const float g = given && args.grad_logprob ? args.grad_logprob[row] * args.scale : 0.0f;
  const float h = kEntropy ? args.grad_entropy[row] * args.scale : 0.0f;
  float w = -g;
  if (args.grad_lse) w += args.grad_lse[row] * args.scale;
  if (kEntropy) w -= h * args.entropy[row];
  const int64_t at = given ? id - args.x.first[r] : -1;  // this rank's column of the given token
#pragma unroll
  for (int v = 0; v < kBackVecs; ++v) {
    const int c = col0 + (v * kThreads + (int)threadIdx.x) * T::kVec;
    if (c >= width) continue;
    float x[T::kVec], d[T::kVec];
    T::widen(raw[v], x);
#pragma unroll
    for (int i = 0; i < T::kVec; ++i) {
      // z rounded first: far out, a fused x * scale - lse is the rounding of lse
      const float logp = x[i] * args.scale - lse;
      const float p = exp2_(logp * kLog2e);
      d[i] = kEntropy ? p * __builtin_fmaf(-h, fmaxf(logp, -150.0f), w) : p * w;
      if (empty) d[i] = 0.0f;
    }
    if (at >= c && at < c + T::kVec) {
#pragma unroll
      for (int i = 0; i < T::kVec; ++i)
        if (at == c + i) d[i] += g;
    }
    store_part<T>(dst + c, width - c, T::round(d));
  }
}

// ---- host -------------------------------------------------------------------

rar_result_t fill_shards(Shards& s, const void* const* logits, const int64_t* widths, const int64_t* strides,
                         int nranks, int64_t rows, int dtype, bool backward) {
  if (nranks < 1 || nranks > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "nranks must be in [1, 64]");
  if (rar_result_t r = check_float_dtype(dtype)) return r;
  if (rows < 0 || rows > kMaxRows) return set_error(RAR_INVALID_ARGUMENT, "rows must be in [0, 2^23]");
  if (!widths) return set_error(RAR_INVALID_ARGUMENT, "widths is NULL");
  const int tile = dtype == RAR_BFLOAT16 ? (backward ? block_tile<BF16>() : wave_tile<BF16>())
                                         : (backward ? block_tile<F32>() : wave_tile<F32>());
  int64_t vocab = 0, tiles = 0;
  for (int r = 0; r < nranks; ++r) {
    if (widths[r] < 0 || widths[r] > (int64_t(1) << 30))
      return set_error(RAR_INVALID_ARGUMENT, "width of rank " + std::to_string(r) + " out of range");
    s.first[r] = (int32_t)vocab;
    s.tile0[r] = (int32_t)tiles;
    vocab += widths[r];
    tiles += (widths[r] + tile - 1) / tile;
    if (vocab > (int64_t(1) << 30)) return set_error(RAR_INVALID_ARGUMENT, "the vocabulary must have at most 2^30 tokens");
    if (rar_result_t e = set_stride(s.stride[r], strides, r, widths[r], rows, "row stride of rank")) return e;
  }
  if (vocab == 0) return set_error(RAR_INVALID_ARGUMENT, "the vocabulary is empty");
  s.first[nranks] = (int32_t)vocab;
  s.tile0[nranks] = (int32_t)tiles;
  s.nranks = nranks;
  if (rows == 0 || !logits) return RAR_SUCCESS;
  const size_t es = (size_t)elem_size(dtype);
  for (int r = 0; r < nranks; ++r) {
    if (widths[r] == 0) continue;
    if (rar_result_t e = check_pointer(logits[r], es, "logits of rank", r)) return e;
    s.ptr[r] = logits[r];
  }
  return RAR_SUCCESS;
}

// How a row is cut: waves of a workgroup, and workgroups.
struct Cut {
  int waves, splits;
};
// 16 waves for each of 256 compute units, at most one for each tile: one
// workgroup of 4, 8 or 16 waves a row where that is enough, else several of 8
// and a join.  Measured (us, by waves x workgroups a row; 131072 tokens bf16,
// no / 20 alternatives): 1 row 8x8 6.6 / 13.3, 16x4 7.4 / 14.1; 104 rows 8x4
// 11.3 / 21.1, 16x1 11.7 / 23.8; 256 rows 16x1 14.1 / 25.5, 8x1 16.2 / 33;
// 512 rows 8x1 24 / 40, 16x1 26 / 47; 4096 rows 4x1 176 / 215, 8x1 173 / 222,
// 16x1 185 / 343.
Cut choose_cut(const Shards& s, int64_t rows, int ntop) {
  const int tiles = s.tile0[s.nranks];
  const int64_t want = std::min<int64_t>(tiles, 4096 / std::max<int64_t>(1, rows));
  Cut c{want > 8 ? 16 : want > 4 ? 8 : 4, 1};
  if (want > 16) {
    c.waves = 8;
    int64_t splits = std::min<int64_t>((want + 7) / 8, kMaxSplits);
    if (ntop) splits = std::min<int64_t>(splits, kCandidates / ntop);
    c.splits = (int)splits;
  }
  return c;
}
// The least logit that is not masked.  fp32's own lowest up to scale 1; above,
// the quotient is within a rounding of it.
float least_logit(float scale) {
  constexpr float kLowest = -std::numeric_limits<float>::max();
  if (scale <= 1.0f) return kLowest;
  float x = kLowest / scale;
  while (!(x * scale >= kLowest)) x = std::nextafter(x, 0.0f);
  for (float y; (y = std::nextafter(x, kLowest)) * scale >= kLowest;) x = y;
  return x;
}
size_t workspace_for(int64_t rows, int splits, int ntop) {
  return splits == 1 ? 0 : (size_t)rows * splits * (16 + 8 * (size_t)ntop);
}

template <class T>
const void* pick_logprobs(bool top, int waves) {
  if (waves == 16)
    return top ? reinterpret_cast<const void*>(&logprobs_kernel<T, true, 16>)
               : reinterpret_cast<const void*>(&logprobs_kernel<T, false, 16>);
  if (waves == 8)
    return top ? reinterpret_cast<const void*>(&logprobs_kernel<T, true, 8>)
               : reinterpret_cast<const void*>(&logprobs_kernel<T, false, 8>);
  return top ? reinterpret_cast<const void*>(&logprobs_kernel<T, true, 4>)
             : reinterpret_cast<const void*>(&logprobs_kernel<T, false, 4>);
}

rar_result_t logprobs_call(const void* const* logits, const int64_t* widths, const int64_t* strides, int nranks,
                           int64_t rows, int dtype, float scale, const int64_t* ids, int ntop, float* logprob,
                           float* entropy, float* lse, int32_t* top_ids, float* top_logprobs, void* workspace,
                           size_t workspace_bytes, void* stream) {
  LogprobsArgs a{};
  if (rar_result_t r = fill_shards(a.x, logits, widths, strides, nranks, rows, dtype, false)) return r;
  if (!(scale > 0.0f) || !std::isfinite(scale) || !std::isfinite(scale * kLog2e))
    return set_error(RAR_INVALID_ARGUMENT, "scale must be positive and finite");
  if (ntop < 0 || ntop > kMaxTop) return set_error(RAR_INVALID_ARGUMENT, "ntop must be in [0, 32]");
  if (rows == 0) return RAR_SUCCESS;
  if (!logits) return set_error(RAR_INVALID_ARGUMENT, "logits is NULL");
  if (!logprob && !entropy && !lse && !ntop) return set_error(RAR_INVALID_ARGUMENT, "no output is asked for");
  const size_t es = (size_t)elem_size(dtype);
  std::vector<Block> reads, writes;
  reads.reserve(nranks + 6);
  writes.reserve(nranks + 6);
  for (int r = 0; r < nranks; ++r)
    reads.push_back({a.x.ptr[r], rows, (int64_t)(widths[r] * es), (int64_t)(a.x.stride[r] * es), "logits"});
  auto out = [&](void* p, size_t align, int64_t bytes, const char* what) -> rar_result_t {
    if (!p) return RAR_SUCCESS;
    if (rar_result_t r = check_pointer(p, align, what)) return r;
    writes.push_back({p, 1, bytes, bytes, what});
    return RAR_SUCCESS;
  };
  if (logprob) {
    if (rar_result_t r = check_pointer(ids, 8, "ids")) return r;
    reads.push_back({ids, 1, rows * 8, rows * 8, "ids"});
  }
  if (ntop) {
    if (rar_result_t r = check_pointer(top_ids, 4, "top_ids")) return r;
    if (rar_result_t r = check_pointer(top_logprobs, 4, "top_logprobs")) return r;
  }
  if (rar_result_t r = out(logprob, 4, rows * 4, "logprob")) return r;
  if (rar_result_t r = out(entropy, 4, rows * 4, "entropy")) return r;
  if (rar_result_t r = out(lse, 4, rows * 4, "lse")) return r;
  if (ntop) {
    if (rar_result_t r = out(top_ids, 4, rows * ntop * 4, "top_ids")) return r;
    if (rar_result_t r = out(top_logprobs, 4, rows * ntop * 4, "top_logprobs")) return r;
  }
  const Cut cut = choose_cut(a.x, rows, ntop);
  a.splits = cut.splits;
  const size_t need = workspace_for(rows, a.splits, ntop);
  if (need) {
    if (workspace_bytes < need)
      return set_error(RAR_INVALID_ARGUMENT, "workspace holds " + std::to_string(workspace_bytes) + " bytes, " +
                                                 std::to_string(need) + " needed");
    if (rar_result_t r = out(workspace, 16, (int64_t)need, "workspace")) return r;
    if (!workspace) return set_error(RAR_INVALID_ARGUMENT, "workspace is NULL");
  }
  if (rar_result_t r = check_blocks(reads, writes)) return r;
  a.ntop = ntop;
  a.scale = scale;
  a.scale2 = scale * kLog2e;
  a.least = least_logit(scale);
  a.ids = ids;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.parts = static_cast<v4f*>(workspace);
  a.keys = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + (size_t)rows * a.splits * 16);
  const bool bf = dtype == RAR_BFLOAT16;
  const void* fn = bf ? pick_logprobs<BF16>(ntop > 0, cut.waves) : pick_logprobs<F32>(ntop > 0, cut.waves);
  if (rar_result_t r = launch_kernel(fn, dim3((unsigned)(rows * a.splits)), dim3(cut.waves * kWaveSize), &a, stream)) return r;
  if (a.splits == 1) return RAR_SUCCESS;
  const void* join_fn = bf ? reinterpret_cast<const void*>(&logprobs_join_kernel<BF16>)
                           : reinterpret_cast<const void*>(&logprobs_join_kernel<F32>);
  return launch_kernel(join_fn, dim3((unsigned)rows), dim3(kThreads), &a, stream);
}

rar_result_t logprobs_backward_call(const void* const* logits, const int64_t* widths, const int64_t* strides,
                                    int nranks, int64_t rows, int dtype, float scale, const int64_t* ids,
                                    const float* lse, const float* entropy, const float* grad_logprob,
                                    const float* grad_entropy, const float* grad_lse, void* const* grads,
                                    const int64_t* grad_strides, void* stream) {
  LogprobsBackwardArgs a{};
  if (rar_result_t r = fill_shards(a.x, logits, widths, strides, nranks, rows, dtype, true)) return r;
  if (!(scale > 0.0f) || !std::isfinite(scale))
    return set_error(RAR_INVALID_ARGUMENT, "scale must be positive and finite");
  if (rows == 0) return RAR_SUCCESS;
  if (!logits || !grads) return set_error(RAR_INVALID_ARGUMENT, "logits or grads is NULL");
  const size_t es = (size_t)elem_size(dtype);
  std::vector<Block> reads, writes;
  reads.reserve(nranks + 6);
  writes.reserve(nranks + 6);
  for (int r = 0; r < nranks; ++r) {
    // in place over its own logits alone: other ranks' are other workgroups'
    reads.push_back({a.x.ptr[r], rows, (int64_t)(widths[r] * es), (int64_t)(a.x.stride[r] * es), "logits",
                     widths[r] ? (int)writes.size() : kNoOutput});
    if (widths[r] == 0) continue;
    if (rar_result_t e = check_pointer(grads[r], es, "gradient of rank", r)) return e;
    if (rar_result_t e = set_stride(a.grad_stride[r], grad_strides, r, widths[r], rows, "gradient row stride of rank")) return e;
    a.grad[r] = grads[r];
    writes.push_back({grads[r], rows, (int64_t)(widths[r] * es), (int64_t)(a.grad_stride[r] * es), "gradient"});
  }
  auto in = [&](const void* p, size_t size, const char* what) -> rar_result_t {
    if (!p) return RAR_SUCCESS;
    if (rar_result_t r = check_pointer(p, size, what)) return r;
    reads.push_back({p, 1, (int64_t)(rows * size), (int64_t)(rows * size), what});
    return RAR_SUCCESS;
  };
  if (!ids || !lse) return set_error(RAR_INVALID_ARGUMENT, "ids or lse is NULL");
  if (!grad_logprob && !grad_entropy && !grad_lse) return set_error(RAR_INVALID_ARGUMENT, "no gradient is given");
  if (grad_entropy && !entropy) return set_error(RAR_INVALID_ARGUMENT, "entropy is NULL");
  if (rar_result_t r = in(ids, 8, "ids")) return r;
  if (rar_result_t r = in(lse, 4, "lse")) return r;
  if (rar_result_t r = in(grad_entropy ? entropy : nullptr, 4, "entropy")) return r;
  if (rar_result_t r = in(grad_logprob, 4, "grad_logprob")) return r;
  if (rar_result_t r = in(grad_entropy, 4, "grad_entropy")) return r;
  if (rar_result_t r = in(grad_lse, 4, "grad_lse")) return r;
  if (rar_result_t r = check_blocks(reads, writes)) return r;
  a.scale = scale;
  a.ids = ids;
  a.lse = lse;
  a.entropy = entropy;
  a.grad_logprob = grad_logprob;
  a.grad_entropy = grad_entropy;
  a.grad_lse = grad_lse;
  const bool bf = dtype == RAR_BFLOAT16;
  const void* fn = bf ? (grad_entropy ? reinterpret_cast<const void*>(&logprobs_backward_kernel<BF16, true>)
                                      : reinterpret_cast<const void*>(&logprobs_backward_kernel<BF16, false>))
                      : (grad_entropy ? reinterpret_cast<const void*>(&logprobs_backward_kernel<F32, true>)
                                      : reinterpret_cast<const void*>(&logprobs_backward_kernel<F32, false>));
  // rows that one grid can hold, launch after launch
  const int64_t tiles = a.x.tile0[nranks];
  for (int64_t row0 = 0, step = std::max<int64_t>(1, kMaxBlocks / tiles); row0 < rows; row0 += step) {
    a.row0 = row0;
    const int64_t blocks = std::min(step, rows - row0) * tiles;
    if (rar_result_t r = launch_kernel(fn, dim3((unsigned)blocks), dim3(kThreads), &a, stream)) return r;
  }
  return RAR_SUCCESS;
}

}  // namespace
}  // namespace rar

extern "C" {

rar_result_t rar_logprobs_workspace(const int64_t* widths, int nranks, int64_t rows, rar_dtype_t dtype, int ntop,
                                    size_t* bytes) {
  return rar::guarded([&]() -> rar_result_t {
    rar::Shards s{};
    if (!bytes) return rar::set_error(RAR_INVALID_ARGUMENT, "bytes is NULL");
    if (rar_result_t r = rar::fill_shards(s, nullptr, widths, nullptr, nranks, rows, dtype, false)) return r;
    if (ntop < 0 || ntop > rar::kMaxTop) return rar::set_error(RAR_INVALID_ARGUMENT, "ntop must be in [0, 32]");
    *bytes = rar::workspace_for(rows, rar::choose_cut(s, rows, ntop).splits, ntop);
    return RAR_SUCCESS;
  });
}

rar_result_t rar_logprobs(const void* const* logits, const int64_t* widths, const int64_t* strides, int nranks,
                          int64_t rows, rar_dtype_t dtype, float scale, const int64_t* ids, int ntop, float* logprob,
                          float* entropy, float* lse, int32_t* top_ids, float* top_logprobs, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return rar::guarded([&] {
    return rar::logprobs_call(logits, widths, strides, nranks, rows, dtype, scale, ids, ntop, logprob, entropy, lse,
                              top_ids, top_logprobs, workspace, workspace_bytes, stream);
  });
}

rar_result_t rar_logprobs_backward(const void* const* logits, const int64_t* widths, const int64_t* strides,
                                   int nranks, int64_t rows, rar_dtype_t dtype, float scale, const int64_t* ids,
                                   const float* lse, const float* entropy, const float* grad_logprob,
                                   const float* grad_entropy, const float* grad_lse, void* const* grads,
                                   const int64_t* grad_strides, void* stream) {
  return rar::guarded([&] {
    return rar::logprobs_backward_call(logits, widths, strides, nranks, rows, dtype, scale, ids, lse, entropy,
                                       grad_logprob, grad_entropy, grad_lse, grads, grad_strides, stream);
  });
}

}  // extern "C"
