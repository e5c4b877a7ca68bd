// adapters.hip -- low-rank adapters of many requests beside a row-parallel
// projection, with the projection's one-shot AllReduce.
//
//   y_t = sum_r P_r[t] + scale_a * B_a (sum_r A_{a,r} x_r[t]),   a = ids[t]
//
// Rank r holds the columns x_r of the input, the partial product P_r of the
// shared projection and its part A_{a,r} of each adapter; tokens with an id
// outside [0, adapters) have no adapter.  Two kernels: `shrink` forms
// h_t = A x_t in fp32, the inner dimension cut into parts over workgroups,
// and `expand` adds up the parts, forms B h, folds the ranks' partials in
// rank order and writes y to every copy, rounded to the payload type once.
//
// Both products are MFMA tiles of 16 x 16.  A tile's tokens may have different
// adapters: the adapters of a tile are taken in turn, with the other tokens'
// rows left out.  An adapter's non-finite weights reach its own tokens only.
// In bf16, h enters expand as the sum of two bf16 numbers (16 bits of it).
//
// Bound by memory: x, the partials and y move once; 2 * rank flops for each
// element of x and y are far below the matrix rate.  Measured (kernels, 4
// ranks, 7168 x 7168, bf16): 4096 tokens of 7 requests, rank 64: shrink 30 us
// (59 MB of x and 40 MB of weights past the L2), expand 108 us (470 MB, 4.4
// TB/s; the one-shot AllReduce moves 512 MiB in 88); 512 tokens, each with one
// of 64 adapters of rank 64: 67 + 77 us (183 MB), where a tile of tokens takes
// one adapter after the other; 104 tokens with 64 adapters of rank 16: 9.8 +
// 9.2 us; 1 token 4.4 + 5.6 us, the time that two dependent launches and their
// chains of loads take.  fp32: 4096 tokens 86 + 199 us, 104 tokens 16.8 + 12.2.
#include "op_common.h"

namespace rar {
namespace {

constexpr int kMaxRank = 128;  // of an adapter
constexpr int kThreads = 256, kWaves = kThreads / kWaveSize;
constexpr int kMaxParts = 16;
constexpr int kRunCols = 64 * kWaves;  // columns of an expand workgroup

struct ShrinkArgs {
  const void* x[kMaxRanks];
  int64_t x_stride[kMaxRanks];
  const void* down[kMaxRanks];   // [adapters][rank][width]
  int32_t width[kMaxRanks];
  int32_t step0[kMaxRanks + 1];  // first step of each rank
  const int64_t* ids;
  float* h;                      // [parts][tokens][rank]
  int64_t tokens;
  int32_t nranks, adapters, rank, parts, slots;
};
struct ExpandArgs {
  const void* partial[kMaxRanks];
  int64_t partial_stride[kMaxRanks];
  void* out[kMaxRanks];
  int64_t out_stride[kMaxRanks];
  const void* up;                // [adapters][outer][rank]
  const int64_t* ids;
  const float* scales;
  const float* h;
  int64_t tokens;
  int64_t run0;                  // first run of the launch
  int32_t nranks, ncopies, adapters, rank, outer, parts, run_tiles;
};

// A step of the inner dimension: 2 vectors for each of the 4 lane groups.
template <class T>
constexpr int step_width() { return 8 * T::kVec; }

// One 16-byte vector of each operand: 32 (bf16) or 16 (fp32) of the inner
// dimension, lane group g = lane / 16 holding places g * kVec ...
template <class T>
__device__ __forceinline__ v4f mma(v4u a, v4u b, v4f c) {
  if constexpr (T::kVec == 8) {
    typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  }
}

// The adapter of a token, or -1.
__device__ __forceinline__ int load_id(const int64_t* ids, int64_t token, int64_t tokens, int adapters) {
  if (token >= tokens) return -1;
  const int64_t id = ids[token];
  return id >= 0 && id < adapters ? (int)id : -1;
}

// h of 16 * kM tokens and one part of the inner dimension, for the adapters
// slot, slot + slots, ... of the tile.  The waves split the part's steps
// between them and their sums meet in LDS.  kN tiles of 16 cover the
// adapter's rank.
//
// Each wave stages a step's operands, 128 bytes of every row, in LDS: a load
// there takes 8 whole lines, while in the MFMA's own layout, where
// neighbouring lanes are different rows, it takes 45 accesses to the cache
// (4096 tokens of 7168, rank 64: 45 us,
// staged 34 us, with all of a step's loads issued together 30 us).
template <class T, int kN, int kM>
__global__ void __launch_bounds__(kThreads) shrink_kernel(ShrinkArgs) {
  const ShrinkArgs& args = kernel_args<ShrinkArgs>();
  constexpr int kStep = step_width<T>();
  constexpr int kLoads = 2 * (kM + kN);  // of 8 rows each
  typedef typename T::bits bits;
  union Lds {
    v4u rows[kWaves][16 * (kM + kN)][9];  // 128 bytes and 16 against bank conflicts
    v4f sums[kWaves][kM][kN][kWaveSize];
  };
  __shared__ Lds lds;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, group = lane >> 4, at = lane & 15;
  const int64_t token0 = (int64_t)blockIdx.x * 16 * kM;
  const int part = blockIdx.y, steps = args.step0[args.nranks];
  const int begin = (int)((int64_t)steps * part / args.parts), end = (int)((int64_t)steps * (part + 1) / args.parts);
  // lane l stands for token l of the tile
  const int id = lane < 16 * kM ? load_id(args.ids, token0 + lane, args.tokens, args.adapters) : -1;
  uint64_t left = __ballot(id >= 0);
  for (int k = 0; left; ++k) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t members = __ballot(id == a);
    left &= ~members;
    if (k % args.slots != (int)blockIdx.z) continue;
    v4f acc[kM][kN];
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int n = 0; n < kN; ++n) acc[m][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    // One step's operands: rows 0 .. 16 kM - 1 are tokens, the rest rows of the
    // adapter's weights.  In the place of other adapters' tokens and of rows
    // past the rank a row that is there is repeated; its results are not
    // written.  So all loads are issued together: each with a condition of its
    // own, they would wait for each other.
    const int first = __builtin_ctzll(members);
    v4u next[kLoads];
    auto load = [&](int step) {
      int r = 0;
      while (r + 1 < args.nranks && args.step0[r + 1] <= step) ++r;
      const int width = args.width[r];
      const int col0 = (step - args.step0[r]) * kStep, col = col0 + lane % 8 * T::kVec;
      const bool full = col0 + kStep <= width;
      const bits* x = static_cast<const bits*>(args.x[r]) + token0 * args.x_stride[r] + col;
      const bits* w = static_cast<const bits*>(args.down[r]) + (int64_t)a * args.rank * width + col;
      auto row_at = [&](int i) {
        const int row = i * 8 + lane / 8;
        if (i < 2 * kM) return x + (bit_of(members, row) ? row : first) * args.x_stride[r];
        const int n = row - 16 * kM;
        return w + (int64_t)(n < args.rank ? n : args.rank - 1) * width;
      };
      if (full) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) next[i] = load_16(row_at(i));
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) next[i] = load_part<T>(row_at(i), width - col, 0);
      }
    };
    __syncthreads();  // the previous adapter's sums have been read
    if (begin + wave < end) load(begin + wave);
    for (int step = begin + wave; step < end; step += kWaves) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) lds.rows[wave][i * 8 + lane / 8][lane % 8] = next[i];
      wave_lds_fence();
      if (step + kWaves < end) load(step + kWaves);  // in flight during the products
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        v4u x[kM];
#pragma unroll
        for (int m = 0; m < kM; ++m) x[m] = lds.rows[wave][m * 16 + at][v * 4 + group];
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const v4u w = lds.rows[wave][(kM + n) * 16 + at][v * 4 + group];
#pragma unroll
          for (int m = 0; m < kM; ++m) acc[m][n] = mma<T>(x[m], w, acc[m][n]);
        }
      }
      wave_lds_fence();
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int n = 0; n < kN; ++n) lds.sums[wave][m][n][lane] = acc[m][n];
    __syncthreads();
    // lane: column (place in the adapter's rank) `at`, rows (tokens) 4 * group + i
    for (int q = wave; q < kM * kN; q += kWaves) {
      const int m = q / kN, n = q % kN;
      v4f s = lds.sums[0][m][n][lane];
#pragma unroll
      for (int o = 1; o < kWaves; ++o) s += lds.sums[o][m][n][lane];
      const int col = n * 16 + at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = m * 16 + 4 * group + i;
        if (col < args.rank && bit_of(members, row))
          args.h[((int64_t)part * args.tokens + token0 + row) * args.rank + col] = s[i];
      }
    }
  }
}

// Place q of h of a token: its parts' sum.  The loads of 8 parts are issued
// together.
__device__ __forceinline__ float sum_parts(const float* h, int64_t stride, int parts) {
  float s = 0.0f;
  for (int p0 = 0; p0 < parts; p0 += 8) {
    float f[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) f[p] = p0 + p < parts ? h[(int64_t)(p0 + p) * stride] : 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) s += f[p];
  }
  return s;
}

// A number as the sum of n of the payload type: fp32 itself, or three of bf16,
// each the leading 8 bits of what is left (toward zero: a finite number's are
// finite).  They have the number's sign, and are not 0 unless it is, or is
// below 2^-93 (2^-40 of it in the place of nothing left): so an infinite
// weight's products with them add up to an infinity, where one with 0 would
// give NaN.
template <class T, int n>
__device__ __forceinline__ void split(float v, float* part) {
  part[0] = v;
  if constexpr (n > 1) {
    const float least = v * 0x1p-40f;  // of an infinity: itself
    part[0] = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
    float left = fabsf(v) <= 3.402823466e+38f ? v - part[0] : 0.0f;  // fp32's largest
#pragma unroll
    for (int f = 1; f < n; ++f) {
      const float head = __uint_as_float(__float_as_uint(left) & 0xFFFF0000u);
      left -= head;
      part[f] = head != 0.0f ? head : least;
    }
  }
}

// y of a run of at most kTiles * 16 tokens x 256 columns, a tile of 16 tokens
// at a time.  The run's h is laid out in LDS first, for bf16 as three bf16
// numbers whose sum is h (4096 x 7168, 4 ranks, both kernels: rank 64, of two
// numbers and 16 bits 131 us, of three 132; rank 128 189 and 193).  In the
// products a wave takes 64 columns, which are the MFMA's rows, and the tokens
// are its columns.  The result passes through LDS, so that the partials and y
// move in pieces of 256 neighbouring columns, four tokens a wave (4096 x 7168,
// 4 ranks, without any adapter, when this was chosen: in the products' own
// layout, 64 bytes a piece, 150 us; 64 columns a piece 104 us, 256 columns 107
// us, and 93 now; 1000 x 5001, whose rows are not aligned: 64 columns a piece
// 41 us, 256 columns 30 us).
// For bf16 ranks up to 32 the registers are held to 128, four workgroups a
// compute unit (both kernels, rank 16: 1000 x 7168 without the bound 42 us,
// with it 39; 4096 x 7168 111.5 and 110.5, at rank 32 112.2 and 112.7).
// Larger ranks lose by it (rank 64 132 us without, 133 with it; 48 137 and
// 141).
template <class T, int kR, int kTiles>  // kR vectors of each lane group cover the adapter's rank
__global__ void __launch_bounds__(kThreads, T::kVec == 8 && kR == 1 ? 4 : 1) expand_kernel(ExpandArgs) {
  const ExpandArgs& args = kernel_args<ExpandArgs>();
  constexpr int kStep = 4 * T::kVec, kVecs = 16 / T::kVec, kBatch = 4;
  constexpr int kRowVecs = 4 * kR + 1;  // of a token's h; one more against bank conflicts
  constexpr int kForms = T::kVec == 8 ? 3 : 1;
  constexpr int kRowLanes = kRunCols / T::kVec;      // threads that move a token's columns
  constexpr int kRows = kWaveSize * T::kVec / kRunCols > 0 ? kWaveSize * T::kVec / kRunCols : 1;  // tokens a wave's vector covers
  static_assert(kRows * kVecs * kWaves == 16, "four waves move a tile");
  typedef typename T::bits bits;
  __shared__ v4u hs[kForms][kTiles * 16][kRowVecs];
  __shared__ v4f turn[16][kRunCols / 4 + 1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, group = lane >> 4, at = lane & 15;
  const int64_t run0 = (args.run0 + blockIdx.y) * args.run_tiles * 16;
  const int first = (int)blockIdx.x * kRunCols;
  const bool full = first + kRunCols <= args.outer;
  const int left_cols = args.outer - first;
  // vector v of a tile: token row + v * kRows, columns col ..
  const int row = wave * kRows * kVecs + lane / kRowLanes, col = lane % kRowLanes * T::kVec;
  v4u p[kBatch][kVecs];
  auto load_partials = [&](int64_t token0, int r0) {
    const bool whole = full && token0 + 16 <= args.tokens;
    auto each = [&](auto load) {
#pragma unroll
      for (int r = 0; r < kBatch; ++r) {
        if (r0 + r < args.nranks) {
          const int64_t stride = args.partial_stride[r0 + r];
          const bits* src = static_cast<const bits*>(args.partial[r0 + r]) + token0 * stride + first;
#pragma unroll
          for (int v = 0; v < kVecs; ++v) p[r][v] = load(src, row + v * kRows, stride);
        }
      }
    };
    const int64_t rows = args.tokens - token0;
    if (whole) {
      each([&](const bits* src, int at_row, int64_t stride) { return load_nt(src + at_row * stride + col); });
    } else if (left_cols >= T::kVec) {
      // Rows and vectors past the end repeat the last ones, which is not used
      // of them but for the part of a vector that is there.
      const int c = col < left_cols - T::kVec ? col : left_cols - T::kVec;
      each([&](const bits* src, int at_row, int64_t stride) {
        return load_nt(src + (at_row < rows ? at_row : 0) * stride + c);
      });
#pragma unroll
      for (int r = 0; r < kBatch; ++r)
#pragma unroll
        for (int v = 0; v < kVecs; ++v) p[r][v] = shift_elements<T>(p[r][v], col - c);
    } else {
      each([&](const bits* src, int at_row, int64_t stride) {
        return load_part<T>(src + at_row * stride + col, at_row < rows ? left_cols - col : 0, 0);
      });
    }
  };
  // A tile's partials are in flight from the end of the tile before.
  load_partials(run0, 0);
  constexpr int kQuads = kR * kStep / 4;  // of a token's h
#pragma unroll 2
  for (int i = threadIdx.x; i < args.run_tiles * 16 * kQuads; i += kThreads) {
    const int t = i / kQuads, q = i % kQuads * 4;
    const int64_t token = run0 + t < args.tokens ? run0 + t : args.tokens - 1;
    const int64_t id = args.ids[token];
    const bool there = run0 + t < args.tokens && id >= 0 && id < args.adapters;
    float h[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (args.rank % 4 == 0) {
      const float* src = args.h + token * args.rank + (q < args.rank ? q : 0);
      for (int p0 = 0; p0 < args.parts; p0 += 4) {
        v4u f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f[j] = load_16(src + (p0 + j < args.parts ? p0 + j : 0) * args.tokens * args.rank);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] += p0 + j < args.parts ? __uint_as_float(f[j][e]) : 0.0f;
      }
    } else {
      for (int e = 0; e < 4; ++e)
        if (there && q + e < args.rank) h[e] = sum_parts(args.h + token * args.rank + q + e, args.tokens * args.rank, args.parts);
    }
    const float scale = there && args.scales ? args.scales[id] : 1.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = there && q + e < args.rank ? h[e] * scale : 0.0f;
    float part[4][kForms];
#pragma unroll
    for (int e = 0; e < 4; ++e) split<T, kForms>(h[e], part[e]);
#pragma unroll
    for (int f = 0; f < kForms; ++f) {
      const float row[4] = {part[0][f], part[1][f], part[2][f], part[3][f]};
      store4<T>(reinterpret_cast<bits*>(hs[f][t]) + q, 4, row);
    }
  }
  const int col0 = first + wave * 64;  // of the wave's products
  int held = -1;                       // the adapter whose weights are in registers
  v4u w[4][kR];
  for (int tile = 0; tile < args.run_tiles; ++tile) {
    const int64_t token0 = run0 + tile * 16;
    if (token0 >= args.tokens) return;
    __syncthreads();  // h is there, and the tile before has been read from `turn`
    const int id = load_id(args.ids, token0 + at, args.tokens, args.adapters);
    uint64_t left = __ballot(id >= 0) & 0xFFFF;
    const bool any = left != 0;
    if (any && id < 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) turn[at][wave * 16 + j * 4 + group] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    while (left) {
      const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
      const bool mine = id == a;
      left &= ~__ballot(mine);
      if (col0 >= args.outer) continue;
      if (a != held) {
        const bits* up = static_cast<const bits*>(args.up) + ((int64_t)a * args.outer + col0 + at) * args.rank + group * T::kVec;
        if (col0 + 64 <= args.outer && args.rank == kR * kStep) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < kR; ++c) w[j][c] = load_16(up + j * 16 * args.rank + c * kStep);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < kR; ++c)
              w[j][c] = load_part<T>(up + j * 16 * args.rank + c * kStep,
                                     col0 + j * 16 + at < args.outer ? args.rank - c * kStep - group * T::kVec : 0, 0);
        }
        held = a;
      }
      v4f acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kR; ++c)
#pragma unroll
        for (int f = 0; f < kForms; ++f) {
          const v4u h = hs[f][tile * 16 + at][c * 4 + group];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = mma<T>(w[j][c], h, acc[j]);
        }
      // token `at`, columns col0 + j * 16 + 4 * group ..
      if (mine) {
#pragma unroll
        for (int j = 0; j < 4; ++j) turn[at][wave * 16 + j * 4 + group] = acc[j];
      }
    }
    __syncthreads();
    float y[16];
    for (int r0 = 0; r0 < args.nranks; r0 += kBatch) {
      if (r0) load_partials(token0, r0);
#pragma unroll
      for (int r = 0; r < kBatch; ++r) {
        if (r0 + r < args.nranks) {
          float f[16];
#pragma unroll
          for (int v = 0; v < kVecs; ++v) T::widen(p[r][v], f + v * T::kVec);
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = r0 + r == 0 ? f[i] : y[i] + f[i];
        }
      }
    }
    if (tile + 1 < args.run_tiles) load_partials(token0 + 16 < args.tokens ? token0 + 16 : token0, 0);
    if (any) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int q = 0; q < T::kVec / 4; ++q) {
          const v4f d = turn[row + v * kRows][col / 4 + q];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[v * T::kVec + q * 4 + i] += d[i];
        }
    }
    const bool whole = full && token0 + 16 <= args.tokens;
    for (int k = 0; k < args.ncopies; ++k) {
      const int64_t stride = args.out_stride[k];
      bits* dst = static_cast<bits*>(args.out[k]) + (token0 + row) * stride + first + col;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const v4u o = T::round(y + v * T::kVec);
        if (whole) store_nt(dst + v * kRows * stride, o);
        else store_part<T>(dst + v * kRows * stride, token0 + row + v * kRows < args.tokens ? left_cols - col : 0, o);
      }
    }
  }
}

// y of one token x kCols columns: for few tokens, which have few neighbours
// with the same adapter.  kLanes lanes take a row of the adapter's weights, a
// vector each, so that a wave reads neighbouring rows whole.
constexpr int kCols = 1024;
template <class T, int kLanes>
__global__ void __launch_bounds__(kThreads) expand_token_kernel(ExpandArgs) {
  const ExpandArgs& args = kernel_args<ExpandArgs>();
  typedef typename T::bits bits;
  constexpr int kRows = kThreads / kLanes, kBatch = 4;
  __shared__ float hs[kLanes * T::kVec];
  __shared__ float delta[kCols];
  const int64_t token = blockIdx.y;
  const int col0 = blockIdx.x * kCols, tid = threadIdx.x;
  const int cols = args.outer - col0 < kCols ? args.outer - col0 : kCols;
  const int mine = cols - tid * 4;  // of this thread's four neighbouring columns
  const int a = load_id(args.ids, token, args.tokens, args.adapters);  // uniform
  float p[kBatch][4];
  auto load_partials = [&](int r0) {
#pragma unroll
    for (int r = 0; r < kBatch; ++r) {
      if (r0 + r < args.nranks) {
        const bits* src = static_cast<const bits*>(args.partial[r0 + r]) + token * args.partial_stride[r0 + r] + col0 + tid * 4;
        load4<T>(src, mine, p[r]);
      }
    }
  };
  load_partials(0);
  float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (a >= 0) {
    if (tid < kLanes * T::kVec)
      hs[tid] = tid < args.rank ? sum_parts(args.h + token * args.rank + tid, args.tokens * args.rank, args.parts) *
                                      (args.scales ? args.scales[a] : 1.0f)
                                : 0.0f;
    __syncthreads();
    const int q = tid % kLanes * T::kVec;
    float h[T::kVec];
#pragma unroll
    for (int i = 0; i < T::kVec; ++i) h[i] = hs[q + i];
    const bits* up = static_cast<const bits*>(args.up) + ((int64_t)a * args.outer + col0) * args.rank + q;
    auto dot = [&](int row, v4u v) {
      float f[T::kVec], s = 0.0f;
      T::widen(v, f);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) s = __builtin_fmaf(f[i], h[i], s);
      s = group_reduce<kLanes>(s, [](float a, float b) { return a + b; });
      if (tid % kLanes == 0) delta[row] = s;
    };
    if (args.rank == kLanes * T::kVec) {
      // no part vectors: 8 loads in flight (rows past the last repeat it)
      constexpr int kBunch = kCols / kRows < 8 ? kCols / kRows : 8;
      for (int row0 = tid / kLanes; row0 < kCols; row0 += kBunch * kRows) {
        v4u v[kBunch];
#pragma unroll
        for (int i = 0; i < kBunch; ++i) {
          const int row = row0 + i * kRows;
          v[i] = load_16(up + (int64_t)(row < cols ? row : cols - 1) * args.rank);
        }
#pragma unroll
        for (int i = 0; i < kBunch; ++i) dot(row0 + i * kRows, v[i]);
      }
    } else {
      for (int row = tid / kLanes; row < kCols; row += kRows)
        dot(row, load_part<T>(up + (int64_t)row * args.rank, row < cols ? args.rank - q : 0, 0));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = delta[tid * 4 + i];
  }
  float y[4];
  for (int r0 = 0; r0 < args.nranks; r0 += kBatch) {
    if (r0) load_partials(r0);
#pragma unroll
    for (int r = 0; r < kBatch; ++r)
      if (r0 + r < args.nranks) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = r0 + r == 0 ? p[r][i] : y[i] + p[r][i];
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] += d[i];
  for (int k = 0; k < args.ncopies; ++k)
    store4<T>(static_cast<bits*>(args.out[k]) + token * args.out_stride[k] + col0 + tid * 4, mine, y);
}

template <class T, int kM>
const void* pick_shrink(int rank) {
  if (rank <= 16) return reinterpret_cast<const void*>(&shrink_kernel<T, 1, kM>);
  if (rank <= 32) return reinterpret_cast<const void*>(&shrink_kernel<T, 2, kM>);
  if (rank <= 64) return reinterpret_cast<const void*>(&shrink_kernel<T, 4, kM>);
  return reinterpret_cast<const void*>(&shrink_kernel<T, 8, kM>);
}
// Token tiles of a run: one follows the other's loads, and more would take the
// place of workgroups (their h is in LDS; 8192 tokens of 7168, rank 64: runs
// of 4 tiles 250 us in all, of 2 242).
constexpr int kRunTiles = 2;
template <class T>
const void* pick_expand(int rank) {
  if (rank <= 4 * T::kVec) return reinterpret_cast<const void*>(&expand_kernel<T, 1, kRunTiles>);
  if (rank <= 8 * T::kVec) return reinterpret_cast<const void*>(&expand_kernel<T, 2, kRunTiles>);
  if constexpr (T::kVec == 4)
    if (rank > 16 * T::kVec) return reinterpret_cast<const void*>(&expand_kernel<T, 8, kRunTiles>);
  return reinterpret_cast<const void*>(&expand_kernel<T, 4, kRunTiles>);
}
template <class T>
const void* pick_expand_token(int rank) {
  if (rank <= T::kVec) return reinterpret_cast<const void*>(&expand_token_kernel<T, 1>);
  if (rank <= 2 * T::kVec) return reinterpret_cast<const void*>(&expand_token_kernel<T, 2>);
  if (rank <= 4 * T::kVec) return reinterpret_cast<const void*>(&expand_token_kernel<T, 4>);
  if (rank <= 8 * T::kVec) return reinterpret_cast<const void*>(&expand_token_kernel<T, 8>);
  if constexpr (T::kVec == 4)
    if (rank > 16 * T::kVec) return reinterpret_cast<const void*>(&expand_token_kernel<T, 32>);
  return reinterpret_cast<const void*>(&expand_token_kernel<T, 16>);
}

// How a call is cut: token tiles and parts of the inner dimension's steps.
struct Cut {
  int m;       // 16-token tiles that a shrink workgroup takes together
  int tiles;   // of 16 * m tokens
  int slots;   // workgroups over which a tile's adapters are dealt
  int parts;   // of the inner dimension
  bool by_token;
  int step0[kMaxRanks + 1];
};
Cut cut_call(const int64_t* widths, int nranks, int64_t tokens, int dtype, int rank) {
  Cut c{};
  const int step = dtype == RAR_BFLOAT16 ? step_width<BF16>() : step_width<F32>();
  for (int r = 0; r < nranks; ++r) c.step0[r + 1] = c.step0[r] + (int)((widths[r] + step - 1) / step);
  // Few tokens: each may have an adapter of its own.  By token the adapter's
  // second matrix is read for every token; in tiles, for every adapter of a
  // tile.  7168 x 7168, 4 ranks, by token / in tiles, us:
  //            rank 16, one adapter each, of 4 requests; rank 64, each, of 4
  //   64 tokens          15 / 37         10 / 14          27 / 36   16 / 17
  //   128                21 / 42         13 / 15          43 / 42   20 / 18
  //   512                55 / 67         28 / 24         140 / 138  46 / 31
  //   1024               90 / 118        43 / 38         256 / 238  81 / 48
  // Which tokens share an adapter is known on the device alone, so the bound
  // is one for both: where each column pair turns, the worse choice costs less
  // than a third.
  c.by_token = tokens * rank <= 8192;
  c.m = c.by_token ? 1 : 2;
  c.tiles = (int)std::max<int64_t>(1, (tokens + 16 * c.m - 1) / (16 * c.m));
  const int want = std::max(1, 512 / c.tiles);
  // (expand_kernel's workgroups read every part again: 1024 x 7168, rank 64, 50
  // us with 16 parts, 45 with 8)
  c.parts = std::min({want, c.by_token ? kMaxParts : kMaxParts / 2, (c.step0[nranks] + kWaves - 1) / kWaves});
  // A workgroup without an adapter ends at once.
  c.slots = c.by_token ? 16 : std::max(1, std::min(16, 2048 / std::max(1, c.tiles * c.parts)));
  return c;
}

rar_result_t check_adapters(const int64_t* widths, int nranks, int64_t tokens, int dtype, int64_t adapters, int rank) {
  if (nranks < 1 || nranks > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "nranks must be in [1, 64]");
  if (rar_result_t r = check_float_dtype(dtype)) return r;
  if (!widths) return set_error(RAR_INVALID_ARGUMENT, "widths is NULL");
  if (tokens < 0 || tokens > (int64_t(1) << 24)) return set_error(RAR_INVALID_ARGUMENT, "tokens must be in [0, 2^24]");
  if (adapters < 1 || adapters > (int64_t(1) << 24))
    return set_error(RAR_INVALID_ARGUMENT, "adapters must be in [1, 2^24]");
  if (rank < 1 || rank > kMaxRank) return set_error(RAR_INVALID_ARGUMENT, "the adapters' rank must be in [1, 128]");
  for (int r = 0; r < nranks; ++r)
    if (widths[r] < 0 || widths[r] > (int64_t(1) << 24))
      return set_error(RAR_INVALID_ARGUMENT, "width of rank " + std::to_string(r) + " must be in [0, 2^24]");
  return RAR_SUCCESS;
}

rar_result_t adapter_call(const void* const* xs, const int64_t* widths, const int64_t* x_strides,
                          const void* const* partials, const int64_t* partial_strides, int nranks, void* const* outs,
                          const int64_t* out_strides, int ncopies, int64_t tokens, int64_t outer, int dtype,
                          const void* const* downs, const void* up, int64_t adapters, int rank, const int64_t* ids,
                          const float* scales, void* workspace, size_t workspace_bytes, void* stream) {
  if (rar_result_t r = check_adapters(widths, nranks, tokens, dtype, adapters, rank)) return r;
  if (ncopies < 1 || ncopies > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "the number of copies must be in [1, 64]");
  if (outer < 1 || outer > (int64_t(1) << 24)) return set_error(RAR_INVALID_ARGUMENT, "outer must be in [1, 2^24]");
  if (tokens == 0) return RAR_SUCCESS;
  if (!xs || !partials || !outs || !downs) return set_error(RAR_INVALID_ARGUMENT, "an array of buffers is NULL");
  const size_t es = (size_t)elem_size(dtype);
  ShrinkArgs s{};
  ExpandArgs e{};
  std::vector<Block> reads, writes;
  reads.reserve(3 * nranks + 4);
  writes.reserve(ncopies);
  auto flat = [](const void* p, int64_t bytes, const char* what) { return Block{p, 1, bytes, bytes, what}; };
  for (int r = 0; r < nranks; ++r) {
    s.width[r] = (int32_t)widths[r];
    if (rar_result_t q = set_stride(s.x_stride[r], x_strides, r, widths[r], tokens, "input row stride of rank")) return q;
    if (widths[r]) {
      if (rar_result_t q = check_pointer(xs[r], es, "input of rank", r)) return q;
      if (rar_result_t q = check_pointer(downs[r], es, "down weights of rank", r)) return q;
      reads.push_back({xs[r], tokens, (int64_t)(widths[r] * es), (int64_t)(s.x_stride[r] * es), "an input"});
      reads.push_back(flat(downs[r], adapters * rank * widths[r] * (int64_t)es, "down weights"));
    }
    s.x[r] = xs[r];
    s.down[r] = downs[r];
    if (rar_result_t q = set_stride(e.partial_stride[r], partial_strides, r, outer, tokens, "partial row stride of rank")) return q;
    if (rar_result_t q = check_pointer(partials[r], es, "partial of rank", r)) return q;
    e.partial[r] = partials[r];
    // the thread that writes an element of y has read it of every partial
    reads.push_back({partials[r], tokens, (int64_t)(outer * es), (int64_t)(e.partial_stride[r] * es), "a partial", kAnyOutput});
  }
  for (int k = 0; k < ncopies; ++k) {
    if (rar_result_t q = set_stride(e.out_stride[k], out_strides, k, outer, tokens, "row stride of output")) return q;
    if (rar_result_t q = check_pointer(outs[k], es, "output", k)) return q;
    e.out[k] = outs[k];
    writes.push_back({outs[k], tokens, (int64_t)(outer * es), (int64_t)(e.out_stride[k] * es), "output"});
  }
  if (rar_result_t q = check_pointer(up, es, "up weights")) return q;
  if (rar_result_t q = check_pointer(ids, 8, "ids")) return q;
  reads.push_back(flat(up, adapters * outer * rank * (int64_t)es, "up weights"));
  reads.push_back(flat(ids, tokens * 8, "ids"));
  if (scales) {
    if (rar_result_t q = check_pointer(scales, 4, "scales")) return q;
    reads.push_back(flat(scales, adapters * 4, "scales"));
  }
  const Cut cut = cut_call(widths, nranks, tokens, dtype, rank);
  const size_t need = (size_t)cut.parts * tokens * rank * 4;
  if (workspace_bytes < need)
    return set_error(RAR_INVALID_ARGUMENT, "workspace holds " + std::to_string(workspace_bytes) + " bytes, " +
                                               std::to_string(need) + " needed");
  if (rar_result_t q = check_blocks(reads, writes)) return q;
  if (need) {
    if (rar_result_t q = check_pointer(workspace, 16, "workspace")) return q;
    // written while the inputs and partials are still to be read, and read
    // while y is written
    const Block scratch = flat(workspace, (int64_t)need, "workspace");
    if (rar_result_t q = check_blocks({scratch}, writes)) return q;
    for (Block& r : reads) r.in_place = kNoOutput;
    if (rar_result_t q = check_blocks(reads, {scratch})) return q;
  }
  for (int r = 0; r <= nranks; ++r) s.step0[r] = cut.step0[r];
  s.ids = e.ids = ids;
  s.h = static_cast<float*>(workspace);
  e.h = s.h;
  s.tokens = e.tokens = tokens;
  s.nranks = e.nranks = nranks;
  s.adapters = e.adapters = (int32_t)adapters;
  s.rank = e.rank = rank;
  s.parts = e.parts = cut.parts;
  s.slots = cut.slots;
  e.up = up;
  e.scales = scales;
  e.ncopies = ncopies;
  e.outer = (int32_t)outer;
  const bool bf = dtype == RAR_BFLOAT16;
  if (cut.parts) {
    const void* fn = cut.m == 1 ? (bf ? pick_shrink<BF16, 1>(rank) : pick_shrink<F32, 1>(rank))
                                : (bf ? pick_shrink<BF16, 2>(rank) : pick_shrink<F32, 2>(rank));
    if (rar_result_t q = launch_kernel(fn, dim3((unsigned)cut.tiles, (unsigned)cut.parts, (unsigned)cut.slots), dim3(kThreads), &s, stream))
      return q;
  }
  if (cut.by_token)
    return launch_kernel(bf ? pick_expand_token<BF16>(rank) : pick_expand_token<F32>(rank),
                         dim3((unsigned)((outer + kCols - 1) / kCols), (unsigned)tokens), dim3(kThreads), &e, stream);
  const void* fn = bf ? pick_expand<BF16>(rank) : pick_expand<F32>(rank);
  // The longer a run, the fewer times weights are loaded, but 8 workgroups for
  // each compute unit come first (4096 tokens: runs of 1 tile 141 us, of 2 133,
  // of 4 140).
  const int64_t cols = (outer + kRunCols - 1) / kRunCols;
  const int tiles = cols * ((tokens + 16 * kRunTiles - 1) / (16 * kRunTiles)) < 2048 ? 1 : kRunTiles;
  const int64_t runs = (tokens + 16 * tiles - 1) / (16 * tiles);
  e.run_tiles = tiles;
  // a grid's second dimension holds 65535 workgroups
  for (int64_t run0 = 0; run0 < runs; run0 += 65535) {
    e.run0 = run0;
    if (rar_result_t q = launch_kernel(fn, dim3((unsigned)cols, (unsigned)std::min<int64_t>(65535, runs - run0)), dim3(kThreads), &e, stream))
      return q;
  }
  return RAR_SUCCESS;
}

}  // namespace
}  // namespace rar

extern "C" {

rar_result_t rar_adapter_workspace(const int64_t* widths, int nranks, int64_t tokens, rar_dtype_t dtype, int rank,
                                   size_t* bytes) {
  return rar::guarded([&]() -> rar_result_t {
    if (!bytes) return rar::set_error(RAR_INVALID_ARGUMENT, "bytes is NULL");
    if (rar_result_t r = rar::check_adapters(widths, nranks, tokens, dtype, 1, rank)) return r;
    *bytes = (size_t)rar::cut_call(widths, nranks, tokens, dtype, rank).parts * tokens * rank * 4;
    return RAR_SUCCESS;
  });
}

rar_result_t rar_adapter_allreduce(const void* const* xs, const int64_t* widths, const int64_t* x_strides,
                                   const void* const* partials, const int64_t* partial_strides, int nranks,
                                   void* const* recvbufs, const int64_t* recv_strides, int nrecv, int64_t tokens,
                                   int64_t outer, rar_dtype_t dtype, const void* const* downs, const void* up,
                                   int64_t adapters, int rank, const int64_t* ids, const float* scales,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  return rar::guarded([&] {
    return rar::adapter_call(xs, widths, x_strides, partials, partial_strides, nranks, recvbufs, recv_strides, nrecv,
                             tokens, outer, dtype, downs, up, adapters, rank, ids, scales, workspace, workspace_bytes,
                             stream);
  });
}

}  // extern "C"
