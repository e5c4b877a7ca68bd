// projection8.hip -- a row-parallel projection in 8-bit integers with its
// AllReduce, and the quantisation of rows split over the ranks.
//
//   quantise    a_t = max over r, k of |x_r[t,k]| / 127,   q_r[t,k] = rint(127 x_r[t,k] / max)
//   projection  y_c[t,d] = residual[t,d] + a_t b_d sum_r sum_k q_r[t,k] w_r[d,k]      c = every copy
//
// The scale of a token, and of a channel d of the weights, holds for all
// ranks: the sum over the ranks' columns is a sum of integers, exact, and the
// result does not depend on how the columns are split.  Sums are int32 (131071
// products of two bytes just fit), to fp32 they are rounded once, then come
// two products, the residual and the rounding to the payload type.
//
// Bound by the weights' bytes for few tokens, by the matrix units for many.
// Measured (kernels, 7168 x 7168, bf16, 4 ranks, 4 copies): 1 token 13.7 us
// (51 MB of weights: 3.8 TB/s), 16 tokens 18.3, 104 tokens 17.9 + 5.9, 256
// tokens 26.6 + 6.0, 1024 tokens 62, 4096 tokens 207 to 235 by the card's clock
// (2030 TOP/s; 177 with one copy, 2380 TOP/s); 8192^3 440 to 510.  A library's product
// of the same integers to int32 alone took 180 us (4096 x 7168 x 7168) and 438
// (8192^3).  Quantisation of 4096 x 7168 bf16 23 to 27 us (88 MB), of 1000 x
// 5001 fp32 10.8.
#include "op_common.h"

#include <numeric>

namespace rar {
namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxOuter = int64_t(1) << 24;
constexpr int64_t kMaxResults = int64_t(1) << 38;
constexpr int64_t kMaxInner = 131071;  // 2^14 a product of two bytes, 2^31 a sum

typedef int32_t v4i __attribute__((ext_vector_type(4)));
typedef int32_t v16i __attribute__((ext_vector_type(16)));

// ---- quantisation --------------------------------------------------------------

struct QuantArgs {
  const void* src[kMaxRanks];
  int64_t src_stride[kMaxRanks];
  int8_t* dst[kMaxRanks];
  int64_t dst_stride[kMaxRanks];
  int64_t width[kMaxRanks];
  float* scales;
  int32_t nranks, pieces;
  int32_t first[kMaxRanks];  // the pieces before a rank's
  uint32_t block0;           // rows in earlier launches
};

// rint(127 x / most), a tie to the even integer as the quotient itself has it.
// The product with 127 / most, 3 roundings, is within 127 * 3 * 2^-24 < 2^-15
// of the quotient: unless it is as close to the middle of two integers, both
// have the same nearest one, which adding 1.5 * 2^23 leaves in the low bits.
// The others are divided in 64 bits, where 127 x is exact and a quotient of
// 24-bit numbers that is no tie is much further from one than the rounding.
// x and most are scaled by a power of two where the product would leave fp32's
// range or lose bits.
struct Quotient {
  float power, factor, most;
  __device__ __forceinline__ explicit Quotient(float m) : most(m) {
    power = m > 0x1p100f ? 0x1p-40f : m < 0x1p-60f ? 0x1p80f : 1.0f;
    factor = 127.0f / (m * power);
  }
  // The integer's low 8 bits are those of the result.
  template <bool kScaled>
  __device__ __forceinline__ uint32_t of(float x, bool* near) const {
    const float r = (kScaled ? x * power : x) * factor, shifted = r + 0x1.8p23f;
    *near = *near || __builtin_fabsf((shifted - 0x1.8p23f) - r) >= 0.5f - 0x1p-15f;
    return __float_as_uint(shifted);
  }
  __device__ __forceinline__ uint32_t divided(float x) const { return (uint32_t)(int32_t)__builtin_rint((double)x * 127.0 / (double)most); }
};

// Memory moves 3 bytes an element in bf16; what the vector units add is kept
// to 8 instructions an element (4096 x 7168: 32 us with a division each, 24 this
// way).
//
// A workgroup takes a token.  Its columns are counted in pieces of 64 vectors,
// each of one rank; a wave keeps its first kKept pieces in registers, loaded
// together, and reads those beyond a second time.
constexpr int kKept = 4;

template <class T>
__global__ void __launch_bounds__(1024) quantize_kernel(QuantArgs) {
  const QuantArgs& args = kernel_args<QuantArgs>();
  __shared__ uint32_t scratch[16];
  const int64_t row = args.block0 + blockIdx.x;
  const int waves = blockDim.x >> 6, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // this lane's elements of a piece: how many are there (0: none)
  auto find = [&](int piece, int* rank, int64_t* e) {
    int r = 0;
    while (r + 1 < args.nranks && args.first[r + 1] <= piece) ++r;
    *rank = r;
    *e = ((int64_t)(piece - args.first[r]) * 64 + lane) * T::kVec;
    return piece < args.pieces ? (int)std::max<int64_t>(0, std::min<int64_t>(args.width[r] - *e, T::kVec)) : 0;
  };
  auto load = [&](int rank, int64_t e, int left) {
    return load_part<T>(static_cast<const typename T::bits*>(args.src[rank]) + row * args.src_stride[rank] + e, left, 0);
  };
  // the largest bits of |x|, which order as the values do, NaN last
  typedef uint16_t v2s __attribute__((ext_vector_type(2)));
  uint32_t most = 0;
  auto look = [&](v4u x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T::kVec == 4) {
        most = std::max(most, x[i] & 0x7FFFFFFFu);
      } else {  // two at a time
        const v2s a = __builtin_bit_cast(v2s, most), b = __builtin_bit_cast(v2s, x[i] & 0x7FFF7FFFu);
        most = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
      }
    }
  };
  v4u kept[kKept];
  int rank[kKept], left[kKept];
  int64_t e[kKept];
#pragma unroll
  for (int j = 0; j < kKept; ++j) {
    left[j] = find(wave + j * waves, &rank[j], &e[j]);
    kept[j] = v4u{0, 0, 0, 0};
    if (left[j] > 0) kept[j] = load(rank[j], e[j], left[j]);
  }
#pragma unroll
  for (int j = 0; j < kKept; ++j) look(kept[j]);
  for (int piece = wave + kKept * waves; piece < args.pieces; piece += waves) {
    int r;
    int64_t at;
    const int n = find(piece, &r, &at);
    if (n > 0) look(load(r, at, n));
  }
  if constexpr (T::kVec == 8) most = std::max(most << 16, most & 0xFFFF0000u);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) most = std::max(most, (uint32_t)__shfl_xor((int)most, d));
  if (lane == 0) scratch[wave] = most;
  __syncthreads();
  for (int w = 0; w < waves; ++w) most = std::max(most, scratch[w]);
  const bool finite = most < 0x7F800000u;
  const float m = __uint_as_float(most);
  if (threadIdx.x == 0) args.scales[row] = finite ? m / 127.0f : __uint_as_float(0x7FC00000u);
  const bool zero = !finite || most == 0;
  const Quotient quotient(m);
  auto store = [&](v4u x, int r, int64_t at, int n) {
    int8_t* out = args.dst[r] + row * args.dst_stride[r] + at;
    float f[T::kVec];
    T::widen(x, f);
    uint32_t b[T::kVec], q[T::kVec / 4];
    bool near = false;
    if (zero) {
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) b[i] = 0;
    } else if (quotient.power == 1.0f) {
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) b[i] = quotient.of<false>(f[i], &near);
    } else {
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) b[i] = quotient.of<true>(f[i], &near);
    }
    if (near) {
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) b[i] = quotient.divided(f[i]);
    }
#pragma unroll
    for (int i = 0; i < T::kVec / 4; ++i)  // the low bytes of four
      q[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x0C0C0400u),
                                   __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0C0C0400u), 0x05040100u);
    if (n == T::kVec) {
      typedef uint32_t u32_user __attribute__((aligned(1)));
      typedef uint64_t u64_user __attribute__((aligned(1)));
      if constexpr (T::kVec == 8) *reinterpret_cast<u64_user*>(out) = (uint64_t)q[T::kVec / 4 - 1] << 32 | q[0];
      else *reinterpret_cast<u32_user*>(out) = q[0];
    } else {
#pragma unroll
      for (int i = 0; i < T::kVec; ++i)
        if (i < n) out[i] = (int8_t)(q[i / 4] >> (8 * (i & 3)));
    }
  };
#pragma unroll
  for (int j = 0; j < kKept; ++j)
    if (left[j] > 0) store(kept[j], rank[j], e[j], left[j]);
  for (int piece = wave + kKept * waves; piece < args.pieces; piece += waves) {
    int r;
    int64_t at;
    const int n = find(piece, &r, &at);
    if (n > 0) store(load(r, at, n), r, at, n);
  }
}

// ---- projection ----------------------------------------------------------------

struct ProjArgs {
  const int8_t* x[kMaxRanks];
  const int8_t* w[kMaxRanks];
  int64_t x_stride[kMaxRanks];
  int64_t w_stride[kMaxRanks];
  int32_t width[kMaxRanks];
  void* dst[kMaxRanks];
  int64_t dst_stride[kMaxRanks];
  const float *x_scales, *w_scales;
  const void* residual;
  int64_t residual_stride;
  int64_t tokens, outer;
  int32_t nranks, ndst;
  int32_t tiles_m, tiles_n;  // of the launch's (last) kind of tile
  int32_t wide_n;            // tiles of 256 channels in front of those of 192
  int32_t steps;  // of kDepth bytes of the inner dimension, each rank's rounded up
  int32_t splits;
  int32_t* partial;  // [splits][tokens][outer]
};

// n bytes (1 to 15) at several places, loaded together, zeros behind: two
// pieces of each that overlap, neither beyond the n bytes.
template <int kCount>
__device__ __forceinline__ void load_ends(const int8_t* const* p, int n, v4u* to) {
  typedef uint32_t v2u_byte __attribute__((ext_vector_type(2), aligned(1)));
  typedef uint32_t u32_byte __attribute__((aligned(1)));
  typedef uint16_t u16_byte __attribute__((aligned(1)));
  v2u lo[kCount], hi[kCount];
#pragma unroll
  for (int i = 0; i < kCount; ++i) lo[i] = hi[i] = v2u{0, 0};
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) lo[i] = *reinterpret_cast<const v2u_byte*>(p[i]), hi[i] = *reinterpret_cast<const v2u_byte*>(p[i] + n - 8);
    // without its first 16 - n bytes, 1 to 8
    const int drop = 16 - n, bits = 8 * (drop & 3);
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      v2u h = drop >= 8 ? v2u{0, 0} : drop >= 4 ? v2u{hi[i][1], 0} : hi[i];
      hi[i] = v2u{__builtin_amdgcn_alignbit(h[1], h[0], bits), h[1] >> bits};
    }
  } else if (n >= 4) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) lo[i][0] = *reinterpret_cast<const u32_byte*>(p[i]), lo[i][1] = *reinterpret_cast<const u32_byte*>(p[i] + n - 4);
#pragma unroll
    for (int i = 0; i < kCount; ++i) lo[i][1] = n > 4 ? lo[i][1] >> (8 * (8 - n)) : 0;
  } else if (n >= 2) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) lo[i][0] = (uint8_t)p[i][0], lo[i][1] = *reinterpret_cast<const u16_byte*>(p[i] + n - 2);
#pragma unroll
    for (int i = 0; i < kCount; ++i) lo[i] = v2u{lo[i][0] | lo[i][1] << (8 * (n - 2)), 0};
  } else {
#pragma unroll
    for (int i = 0; i < kCount; ++i) lo[i][0] = (uint8_t)p[i][0];
  }
#pragma unroll
  for (int i = 0; i < kCount; ++i) to[i] = v4u{lo[i][0], lo[i][1], hi[i][0], hi[i][1]};
}

// 16 bytes of a row from p on, n (1 or more) of them there and zeros behind.
__device__ __forceinline__ v4u load_bytes(const int8_t* p, int n) {
  typedef uint32_t v4u_byte __attribute__((ext_vector_type(4), aligned(1)));
  if (n >= 16) return *reinterpret_cast<const v4u_byte*>(p);
  v4u r;
  load_ends<1>(&p, n, &r);
  return r;
}

// 16 bytes without the first n (0 or more), zeros behind.
__device__ __forceinline__ v4u shift_bytes(v4u v, int n) {
  const int bits = 8 * (n & 3);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_alignbit(i < 3 ? v[i + 1] : 0, v[i], bits);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = n & 4 ? (i < 3 ? v[i + 1] : 0) : v[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = n & 8 ? (i < 2 ? v[i + 2] : 0) : v[i];
  return n < 16 ? v : v4u{0, 0, 0, 0};
}

constexpr int kDepth = 128;  // bytes of the inner dimension that a step has

// The results of token m, channels n ... n + left - 1 (up to T::kVec), from
// their integer sums.
template <class T>
__device__ __forceinline__ void finish(const ProjArgs& args, int64_t m, int64_t n, int left, const int32_t* sum, const float* ws) {
  const float xs = args.x_scales[m];
  float f[T::kVec];
#pragma unroll
  for (int e = 0; e < T::kVec; ++e) f[e] = (float)sum[e] * xs * ws[e];
  if (args.residual) {
    float g[T::kVec];
    T::widen(load_part<T>(static_cast<const typename T::bits*>(args.residual) + m * args.residual_stride + n, left, 0), g);
#pragma unroll
    for (int e = 0; e < T::kVec; ++e) f[e] += g[e];
  }
  const v4u y = T::round(f);
  for (int c = 0; c < args.ndst; ++c) store_part<T>(static_cast<typename T::bits*>(args.dst[c]) + m * args.dst_stride[c] + n, left, y);
}
// The scales of channels n ... n + left - 1.
template <class T>
__device__ __forceinline__ void load_scales(const ProjArgs& args, int64_t n, int left, float* ws) {
#pragma unroll
  for (int v = 0; v < T::kVec; v += 4) load4<F32>(reinterpret_cast<const uint32_t*>(args.w_scales + n + v), left - v, ws + v);
}
__device__ __forceinline__ void store_words(int32_t* p, int n, v4i v) {
  typedef int32_t v4i_user __attribute__((ext_vector_type(4), aligned(4)));
  if (n >= 4) {
    *reinterpret_cast<v4i_user*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ v4i load_words(const int32_t* p, int n) {
  typedef int32_t v4i_user __attribute__((ext_vector_type(4), aligned(4)));
  if (n >= 4) return *reinterpret_cast<const v4i_user*>(p);
  v4i v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < n) v[i] = p[i];
  return v;
}

// Tile (n, m) of workgroup b, of tiles_n x tiles_m; false: none.  Workgroups
// go to the 8 XCDs in turn: each XCD gets a run of tiles, in which any 32 that
// follow each other, which it runs at a time, share the operands of 8 x 4
// (8192^3: 496 -> 467 us against m fastest).
__device__ __forceinline__ bool tile_of(int64_t b, int64_t tiles_m, int64_t tiles_n, int64_t* n, int64_t* m) {
  const int64_t tiles = tiles_m * tiles_n, tile = (b & 7) * ((tiles + 7) / 8) + (b >> 3);
  if (tile >= tiles) return false;
  const int64_t group = tile / (4 * tiles_m), in_group = tile - group * 4 * tiles_m;
  const int columns = (int)std::min<int64_t>(4, tiles_n - group * 4);
  *m = in_group / columns;
  *n = group * 4 + in_group % columns;
  return true;
}

// 16 bytes a lane from base + offset to LDS, to 16 * lane behind `to` (both the
// same in all lanes).  The
// caller waits for it (vmcnt) before a barrier.
__device__ __forceinline__ void to_lds(const int8_t* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(to)),
               "v"(offset), "s"(row_at(reinterpret_cast<const char*>(base), 0))
               : "memory");
}

// A workgroup's tile: kWN x kWM waves, each with kFN x kFM products of 32
// channels x 32 tokens.  The operands of a step are in LDS, rows of 128 bytes
// whose 16-byte pieces are swapped by row so that the lanes of a read meet
// different banks (none conflicted in 8192^3).  They go there from memory
// directly, kStages - 1 steps ahead; through registers the tile of 128 x 128
// took 640 us where this takes 520.
//
// A wave of 64 tokens x 128 channels reads 6 fragments for 8 products, 192 KB a
// step of 256 x 256, 1500 of its 2048 cycles of products at LDS's rate; with 128
// x 128 a wave, 4 waves and so none to hide behind, 4096 tokens took 292 us
// where this took 244.  Fragments are read a quarter of a step ahead: without
// it 4096 tokens took 224 us with one copy, with it 202.
template <class T, int kWN, int kWM, int kFN, int kFM, int kStages>
struct Tile {
  static constexpr int kWaves = kWN * kWM, kThreads = 64 * kWaves;
  static constexpr int kN = kWN * kFN * 32, kM = kWM * kFM * 32;  // channels, tokens
  static constexpr int kLoadsW = kN * 8 / kThreads, kLoadsX = kM * 8 / kThreads, kLoads = kLoadsW + kLoadsX;
  static constexpr int kStage = (kN + kM) * kDepth;
  static constexpr int kPitch = kFN * 32 + 4;  // floats of a result's row: rows start on different banks
  static constexpr int kOut = kWaves * 32 * kPitch * 4;
  static constexpr int kLds = kStages * kStage > kOut ? kStages * kStage : kOut;

  static __device__ __forceinline__ void run(const ProjArgs& args, int8_t* lds, int64_t n0, int64_t m0, int split) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    v16i acc[kFN][kFM];
#pragma unroll
    for (int i = 0; i < kFN; ++i)
#pragma unroll
      for (int j = 0; j < kFM; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[i][j][k] = 0;

    // the next step to load: rank, its inner offset, this lane's rows there
    // (from the tile's first row on; beyond the last row, the last row again)
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t*)lds;
    const int row0 = wave * 8 + (lane >> 3), chunk = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));
    const int last_w = (int)std::min<int64_t>(args.outer - n0, kN) - 1, last_x = (int)std::min<int64_t>(args.tokens - m0, kM) - 1;
    int rank = 0, k0 = 0;
    const int8_t *w0 = nullptr, *x0 = nullptr;
    uint32_t ow[kLoadsW], ox[kLoadsX];
    auto begin_rank = [&] {
      w0 = args.w[rank] + n0 * args.w_stride[rank];
      x0 = args.x[rank] + m0 * args.x_stride[rank];
#pragma unroll
      for (int i = 0; i < kLoadsW; ++i) ow[i] = (uint32_t)std::min(row0 + i * 8 * kWaves, last_w) * (uint32_t)args.w_stride[rank] + chunk * 16;
#pragma unroll
      for (int i = 0; i < kLoadsX; ++i) ox[i] = (uint32_t)std::min(row0 + i * 8 * kWaves, last_x) * (uint32_t)args.x_stride[rank] + chunk * 16;
    };
    auto next = [&] {
      k0 += kDepth;
      if (k0 >= args.width[rank] && rank + 1 < args.nranks) {
        k0 = 0;
        ++rank;
        begin_rank();
      }
    };
    auto load_step = [&](int stage) {
      const int left = args.width[rank] - k0;
      if (left >= kDepth) {
#pragma unroll
        for (int i = 0; i < kLoadsW; ++i) to_lds(w0 + k0, ow[i], lds0 + stage * kStage + (i * kWaves + wave) * 1024);
#pragma unroll
        for (int i = 0; i < kLoadsX; ++i) to_lds(x0 + k0, ox[i], lds0 + stage * kStage + kN * kDepth + (i * kWaves + wave) * 1024);
      } else {  // a rank's last bytes, zeros behind
        const int mine = left - chunk * 16;
        auto from = [&](int i) { return i < kLoadsW ? w0 + k0 + ow[i < kLoadsW ? i : 0] : x0 + k0 + ox[i < kLoadsW ? 0 : i - kLoadsW]; };
        auto to = [&](int i) { return stage * kStage + ((i < kLoadsW ? i * kWaves : kN / 8 + (i - kLoadsW) * kWaves) + wave) * 1024; };
        if (mine >= 16) {
#pragma unroll
          for (int i = 0; i < kLoads; ++i) to_lds(i < kLoadsW ? w0 + k0 : x0 + k0, i < kLoadsW ? ow[i < kLoadsW ? i : 0] : ox[i < kLoadsW ? 0 : i - kLoadsW], lds0 + to(i));
        } else {
          constexpr int kGroup = kLoads > 6 ? 1 : kLoads;  // together as far as registers go
#pragma unroll
          for (int g = 0; g < kLoads; g += kGroup) {
            const int8_t* p[kGroup];
            v4u some[kGroup];
#pragma unroll
            for (int i = 0; i < kGroup; ++i) p[i] = from(g + i), some[i] = v4u{0, 0, 0, 0};
            if (mine > 0) load_ends<kGroup>(p, left & 15, some);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) *reinterpret_cast<v4u*>(&lds[to(g + i) + lane * 16]) = some[i];
          }
        }
      }
      next();
    };
    const int r = lane & 31, wn = (wave % kWN) * kFN * 32, wm = (wave / kWN) * kFM * 32;
    v4i wf[2][kFN], xf[2][kFM];
    auto read_fragments = [&](int stage, int s, int to) {
      // 32 rows apart the swizzle is the same
      const int at = r * kDepth + (((s * 2 + (lane >> 5)) ^ (r >> 1 & 7)) << 4);
      const int8_t* tw = &lds[stage * kStage + wn * kDepth + at];
      const int8_t* tx = &lds[stage * kStage + (kN + wm) * kDepth + at];
#pragma unroll
      for (int i = 0; i < kFN; ++i) wf[to][i] = *reinterpret_cast<const v4i*>(tw + i * 32 * kDepth);
#pragma unroll
      for (int j = 0; j < kFM; ++j) xf[to][j] = *reinterpret_cast<const v4i*>(tx + j * 32 * kDepth);
    };
    auto multiply = [&](int from) {
#pragma unroll
      for (int i = 0; i < kFN; ++i)
#pragma unroll
        for (int j = 0; j < kFM; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[from][i], xf[from][j], acc[i][j], 0, 0, 0);
    };
    // A quarter of a step is multiplied while the next one's fragments are
    // read.  The workgroup meets before the last quarter: then no wave reads
    // the step any more, its place takes the step kStages further on, and the
    // next one is there.  Loads to LDS arrive in order: all but the youngest
    // kStages - 2 steps' have when as many are outstanding at most.  (A rank's
    // last step has as many, or bytes that come through registers: then what
    // was issued before has arrived when they are stored.)
    auto meet = [](bool all) {
      if (kStages == 2 || all) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kStages - 2) * kLoads) : "memory");
      __builtin_amdgcn_s_barrier();
    };
    const int begin = (int)((int64_t)args.steps * split / args.splits), steps = (int)((int64_t)args.steps * (split + 1) / args.splits) - begin;
    if (steps > 0) {
      k0 = begin * kDepth;
      for (int n; k0 >= (n = (args.width[rank] + kDepth - 1) / kDepth * kDepth); ++rank) k0 -= n;
      begin_rank();
      load_step(0);
#pragma unroll
      for (int i = 1; i < kStages; ++i)
        if (i < steps) load_step(i);
      if (steps >= kStages) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kStages - 1) * kLoads) : "memory");
      else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      read_fragments(0, 0, 0);
    }
    int stage = 0;
    for (int step = 0; step < steps; ++step) {
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        read_fragments(stage, s + 1, (s + 1) & 1);
        multiply(s & 1);
#pragma unroll
        for (int g = 0; g < kFN + kFM && g < kFN * kFM; ++g) {  // one read, one product
          __builtin_amdgcn_sched_group_barrier(0x100, kFN * kFM < kFN + kFM ? 2 : 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        }
      }
      meet(step + kStages > steps);
      const int after = stage + 1 == kStages ? 0 : stage + 1;
      if (step + kStages < steps) load_step(stage);
      if (step + 1 < steps) read_fragments(after, 0, 0);
      multiply(1);
      stage = after;
    }
    // Out through LDS, 32 tokens of a wave at a time, so that its rows are
    // completed and written as whole lines.
    __syncthreads();
    constexpr int kLanes = kFN * 32 / T::kVec, kRows = 64 / kLanes;  // lanes of a row, rows at a time
    int32_t* own = reinterpret_cast<int32_t*>(lds) + wave * 32 * kPitch;
    const int column = lane % kLanes * T::kVec;
    const int64_t n = n0 + wn + column;
    const int left = lane < kLanes * kRows ? (int)std::max<int64_t>(0, std::min<int64_t>(T::kVec, args.outer - n)) : 0;
    float ws[T::kVec];
    load_scales<T>(args, n, left, ws);
#pragma unroll
    for (int j = 0; j < kFM; ++j) {
#pragma unroll
      for (int i = 0; i < kFN; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          // lane l has token l & 31 and channels 8 q + 4 (l >> 5) + 0..3
          v4i f;
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = acc[i][j][4 * q + e];
          *reinterpret_cast<v4i*>(&own[(lane & 31) * kPitch + i * 32 + 8 * q + 4 * (lane >> 5)]) = f;
        }
      wave_lds_fence();
#pragma unroll
      for (int it = 0; it < (32 + kRows - 1) / kRows; ++it) {
        const int row = it * kRows + lane / kLanes;
        const int64_t m = m0 + wm + j * 32 + row;
        if (row >= 32 || m >= args.tokens || left == 0) continue;
        int32_t sum[T::kVec];
#pragma unroll
        for (int h = 0; h < T::kVec; h += 4) {
          const v4i v = *reinterpret_cast<const v4i*>(&own[row * kPitch + column + h]);
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[h + e] = v[e];
          if (args.splits > 1) store_words(args.partial + (split * args.tokens + m) * args.outer + n + h, left - h, v);
        }
        if (args.splits == 1) finish<T>(args, m, n, left, sum, ws);
      }
      wave_lds_fence();
    }
  }
};

// 256 x 256: the first wide_n columns of tiles, as many as make whole rounds
// of the 256 CUs; the others 192 channels wide where that leaves fewer CUs idle
// (4096 x 7168 x 7168, one copy: 448 tiles of 256 take two rounds, 202 us; 256
// of them and 256 of 192 take 1.75, 177 us).
template <class T>
__global__ void __launch_bounds__(512, 1) big_tiles_kernel(ProjArgs) {
  typedef Tile<T, 2, 4, 4, 2, 2> Wide;
  typedef Tile<T, 2, 4, 3, 2, 2> Narrow;
  const ProjArgs& args = kernel_args<ProjArgs>();
  __shared__ __attribute__((aligned(16))) int8_t lds[Wide::kLds > Narrow::kLds ? Wide::kLds : Narrow::kLds];
  int64_t n, m;
  const int64_t wide = (args.tiles_m * args.wide_n + 7) / 8 * 8;
  if (blockIdx.x < wide) {
    if (tile_of(blockIdx.x, args.tiles_m, args.wide_n, &n, &m)) Wide::run(args, lds, n * 256, m * 256, 0);
  } else {
    if (tile_of(blockIdx.x - wide, args.tiles_m, args.tiles_n, &n, &m)) Narrow::run(args, lds, args.wide_n * 256 + n * 192, m * 256, 0);
  }
}

// Fewer tiles than CUs: `splits` workgroups a tile, each with a part of the
// inner dimension, and sum_kernel behind them.
template <class T, int kWN, int kWM, int kFN, int kFM, int kStages>
__global__ void __launch_bounds__(64 * kWN * kWM) tiles_kernel(ProjArgs) {
  typedef Tile<T, kWN, kWM, kFN, kFM, kStages> Own;
  const ProjArgs& args = kernel_args<ProjArgs>();
  __shared__ __attribute__((aligned(16))) int8_t lds[Own::kLds];
  int64_t n, m;
  if (tile_of(blockIdx.x, args.tiles_m, args.tiles_n, &n, &m)) Own::run(args, lds, n * Own::kN, m * Own::kM, blockIdx.y);
}

// The sums over the splits, a vector of a token's results a thread.
template <class T>
__global__ void __launch_bounds__(256) sum_kernel(ProjArgs) {
  const ProjArgs& args = kernel_args<ProjArgs>();
  const int64_t m = blockIdx.y, n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * T::kVec;
  if (n >= args.outer) return;
  const int left = (int)std::min<int64_t>(T::kVec, args.outer - n);
  const int32_t* p = args.partial + m * args.outer + n;
  int32_t sum[T::kVec];
#pragma unroll
  for (int e = 0; e < T::kVec; ++e) sum[e] = 0;
#pragma unroll 4
  for (int s = 0; s < args.splits; ++s)
#pragma unroll
    for (int h = 0; h < T::kVec; h += 4) {
      const v4i v = load_words(p + s * args.tokens * args.outer + h, left - h);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[h + e] += v[e];
    }
  float ws[T::kVec];
  load_scales<T>(args, n, left, ws);
  finish<T>(args, m, n, left, sum, ws);
}

// Up to 16 tokens: a workgroup takes 16 channels; its 8 waves share the inner
// dimension, 64 bytes at a time, and read both operands into registers.
constexpr int kFewTokens = 16;
template <class T>
__global__ void __launch_bounds__(512, 4) few_kernel(ProjArgs) {
  // Pieces whose loads are issued together: the 14 that a wave has of 7168 columns
  // are two batches (13.7 us; in batches of 4 15.3, of 14 17.9).  Measured there
  // alone: 4096 columns take two batches too, with 6 of the second's 7 loads for
  // nothing (14.4), 8192 three (18.0).
  constexpr int kBatch = 7;
  const ProjArgs& args = kernel_args<ProjArgs>();
  __shared__ __attribute__((aligned(16))) int32_t sums[8][kFewTokens][16 + 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16, row = std::min<int64_t>(n0 + (lane & 15), args.outer - 1);
  const int tokens = (int)args.tokens, part = (lane >> 4) * 16;
  const int token = std::min(lane & 15, tokens - 1);
  v4i acc = {0, 0, 0, 0};
  // pieces of 64 bytes are counted through the ranks; this wave's next one
  int r = 0, k = wave * 64;
  auto settle = [&] {
    while (r < args.nranks && k >= args.width[r]) k -= (args.width[r] + 63) & ~63, ++r;
  };
  settle();
  while (r < args.nranks) {
    v4u a[kBatch], b[kBatch];
    int drop[kBatch];  // bytes in front of the lane's part (from 16 on: nothing is there)
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int rank = std::min(r, args.nranks - 1), width = args.width[rank];
      const int8_t* w = args.w[rank] + row * args.w_stride[rank];
      const int8_t* x = args.x[rank] + token * args.x_stride[rank];
      if (width >= 16) {  // a part beyond the row's end is read where whole ones end, and shifted
        const int at = r < args.nranks ? std::min(k + part, width - 16) : 0;
        drop[i] = r < args.nranks ? k + part - at : 16;
        a[i] = load_bytes(w + at, 16);
        b[i] = load_bytes(x + at, 16);
      } else {
        drop[i] = r < args.nranks && part == 0 ? 0 : 16;
        a[i] = load_bytes(w, width);
        b[i] = load_bytes(x, width);
      }
      k += 8 * 64;
      settle();
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (__ballot(drop[i] > 0)) a[i] = shift_bytes(a[i], drop[i]), b[i] = shift_bytes(b[i], drop[i]);
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a[i]), __builtin_bit_cast(v4i, b[i]), acc, 0, 0, 0);
    }
  }
  // lane l has token l & 15 and channels 4 (l >> 4) + 0..3
  *reinterpret_cast<v4i*>(&sums[wave][lane & 15][4 * (lane >> 4)]) = acc;
  __syncthreads();
  constexpr int kLanes = 16 / T::kVec;  // threads of a token
  const int m = threadIdx.x / kLanes, column = threadIdx.x % kLanes * T::kVec;
  const int left = (int)std::min<int64_t>(T::kVec, args.outer - n0 - column);
  if (m >= tokens || left <= 0) return;
  int32_t sum[T::kVec];
#pragma unroll
  for (int e = 0; e < T::kVec; ++e) sum[e] = 0;
#pragma unroll
  for (int v = 0; v < 8; ++v)
#pragma unroll
    for (int h = 0; h < T::kVec; h += 4) {
      const v4i part_sum = *reinterpret_cast<const v4i*>(&sums[v][m][column + h]);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[h + e] += part_sum[e];
    }
  float ws[T::kVec];
  load_scales<T>(args, n0 + column, left, ws);
  finish<T>(args, m, n0 + column, left, sum, ws);
}

// Rows that do not begin on multiples of 16 bytes, laid out so that they do;
// 16 bytes a thread.
struct AlignArgs {
  const int8_t* src[kMaxRanks];
  int64_t stride[kMaxRanks];
  int8_t* dst[kMaxRanks];
  int32_t first[kMaxRanks + 1];  // workgroups before a rank's
  int32_t width[kMaxRanks];
  int64_t rows;
  int32_t nranks;
  uint32_t block0;  // workgroups in earlier launches
};
__global__ void __launch_bounds__(256) align_kernel(AlignArgs) {
  const AlignArgs& args = kernel_args<AlignArgs>();
  const int block = (int)(args.block0 + blockIdx.x);
  int i = 0;
  while (i + 1 < args.nranks && args.first[i + 1] <= block) ++i;
  const int width = args.width[i], pieces = (width + 15) / 16;
  const int64_t at = (int64_t)(block - args.first[i]) * 256 + threadIdx.x, row = at / pieces;
  if (row >= args.rows) return;
  const int k = (int)(at - row * pieces) * 16;
  *reinterpret_cast<v4u*>(args.dst[i] + at * 16) = load_bytes(args.src[i] + row * args.stride[i] + k, width - k);
}

// ---- host --------------------------------------------------------------------

rar_result_t check_widths(const int64_t* widths, int nranks, int64_t* total) {
  if (nranks < 1 || nranks > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "nranks must be in [1, 64]");
  if (!widths) return set_error(RAR_INVALID_ARGUMENT, "widths is NULL");
  *total = 0;
  for (int r = 0; r < nranks; ++r)
    if (widths[r] < 0 || (*total += widths[r]) > kMaxInner)
      return set_error(RAR_INVALID_ARGUMENT, "the widths must not be negative and at most 131071 in all");
  return RAR_SUCCESS;
}

rar_result_t quantize(const void* const* xs, const int64_t* widths, const int64_t* x_strides, int nranks, int64_t rows, int dtype,
                      int8_t* const* quantized, const int64_t* q_strides, float* scales, void* stream) {
  int64_t total;
  if (rar_result_t r = check_widths(widths, nranks, &total)) return r;
  if (rar_result_t r = check_float_dtype(dtype)) return r;
  if (rows < 0 || rows > kMaxTokens) return set_error(RAR_INVALID_ARGUMENT, "rows must be in [0, 2^24]");
  if (rows == 0) return RAR_SUCCESS;
  if (!xs || !quantized) return set_error(RAR_INVALID_ARGUMENT, "an array of buffers is NULL");
  QuantArgs a{};
  const int64_t es = elem_size(dtype);
  std::vector<Block> reads, writes;
  reads.reserve(nranks);
  writes.reserve(nranks + 1);
  for (int r = 0; r < nranks; ++r) {
    a.width[r] = widths[r];
    if (rar_result_t e = set_stride(a.src_stride[r], x_strides, r, widths[r], rows, "input stride")) return e;
    if (rar_result_t e = set_stride(a.dst_stride[r], q_strides, r, widths[r], rows, "output stride")) return e;
    if (widths[r] == 0) continue;
    if (rar_result_t e = check_pointer(xs[r], es, "input", r)) return e;
    if (rar_result_t e = check_pointer(quantized[r], 1, "output", r)) return e;
    a.src[r] = xs[r];
    a.dst[r] = quantized[r];
    reads.push_back({xs[r], rows, widths[r] * es, a.src_stride[r] * es, "an input"});
    writes.push_back({quantized[r], rows, widths[r], a.dst_stride[r], "output"});
  }
  if (rar_result_t r = check_pointer(scales, 4, "scales")) return r;
  writes.push_back({scales, 1, rows * 4, rows * 4, "scales"});
  if (rar_result_t r = check_blocks(reads, writes)) return r;
  a.scales = scales;
  a.nranks = nranks;
  const void* fn = dtype == kFloat32 ? reinterpret_cast<const void*>(&quantize_kernel<F32>) : reinterpret_cast<const void*>(&quantize_kernel<BF16>);
  const int piece = 64 * (dtype == kFloat32 ? F32::kVec : BF16::kVec);
  for (int r = 0; r < nranks; ++r) {
    a.first[r] = a.pieces;
    a.pieces += (int32_t)((widths[r] + piece - 1) / piece);
  }
  // as many waves as the device holds (8192), a wave for every kKept pieces
  const int64_t most = std::max<int64_t>((a.pieces + kKept - 1) / kKept, 8192 / rows);
  const int waves = (int)std::max<int64_t>(1, std::min<int64_t>({most, a.pieces, 16}));
  return launch_groups(fn, rows, 64 * waves, &a, &a.block0, stream);
}

rar_result_t check_sizes(int64_t tokens, int64_t outer, int dtype) {
  if (rar_result_t r = check_float_dtype(dtype)) return r;
  if (tokens < 0 || tokens > kMaxTokens) return set_error(RAR_INVALID_ARGUMENT, "tokens must be in [0, 2^24]");
  if (outer < 1 || outer > kMaxOuter) return set_error(RAR_INVALID_ARGUMENT, "outer must be in [1, 2^24]");
  return RAR_SUCCESS;
}

// The kinds of kernel, and which a call takes, by how the tiles fill the CUs.
// Measured, us (7168 x 7168, bf16, 1 copy unless said):
//   up to 16 tokens kFew (16: 18.9, 4 copies); of two fragments it took 23.9 for
//     32, where k64x128 takes 13.8 + 5.4
//   up to 64 k64x128 (50: 13.0 + 4.3; k128x64 14.7 + 4.3)
//   from 160 tiles of 256 x 256 on kBig (1536: 168 tiles 76, 128 x 128 96; 1024:
//     112 tiles 70, 128 x 128 58)
//   from 300 tiles of 128 x 128 on those (768: 336 tiles 50, 128 x 64 63; 512:
//     224 tiles 44, 128 x 64 37)
//   else k128x64.
// Two workgroups a CU of the smallest tiles share the inner dimension where
// tiles are fewer (104, 4 copies: whole 31.6, in 4 parts 16.0 + 5.8; 256: whole
// 30.7, in 2 parts 24.1 + 4.9).  So above 256 tiles nothing is divided, and tiles
// of 128 x 128 never are: 1000 x 5001 x 2051 in fp32 is 264 tiles of 42 steps, 40 us.
// The limits are those of 7168 x 7168; other sizes have not been measured for them.
enum { kFew, kBig, k128x128, k64x128, k128x64 };
struct Plan {
  int kind, splits = 1;
  int64_t align_x = 0, align_w = 0, partial = 0;  // bytes of workspace, in this order
};
int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

Plan plan_of(const int64_t* widths, int nranks, int64_t tokens, int64_t outer, bool align_x, bool align_w) {
  Plan p;
  int64_t steps = 0, padded = 0;
  for (int r = 0; r < nranks; ++r) steps += (widths[r] + kDepth - 1) / kDepth, padded += round_up(widths[r], 16);
  auto tiles = [&](int64_t m, int64_t n) { return (tokens + m - 1) / m * ((outer + n - 1) / n); };
  if (tokens <= kFewTokens) p.kind = kFew;
  else if (tokens <= 64) p.kind = k64x128;
  else if (tiles(256, 256) >= 160) p.kind = kBig;
  else if (tiles(128, 128) >= 300) p.kind = k128x128;
  else p.kind = k128x64;
  if (p.kind == kFew) return p;
  const int64_t small = p.kind == k64x128 ? tiles(64, 128) : tiles(128, 64);
  if (p.kind == k64x128 || p.kind == k128x64) p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({512 / small, steps / 6, 16}));
  if (align_x && padded) p.align_x = round_up(tokens * padded, 256);
  if (align_w && padded) p.align_w = round_up(outer * padded, 256);
  if (p.splits > 1) p.partial = round_up(p.splits * tokens * outer * 4, 256);
  return p;
}
// Whether tiles read an operand as it is: rows on multiples of 16 bytes, with
// offsets of 32 bits within a tile.  One row has no use for its stride.
bool is_aligned(const int8_t* p, int64_t stride, int64_t rows) {
  if (rows == 1) stride = 0;
  return ((reinterpret_cast<uintptr_t>(p) | stride) & 15) == 0 && stride < (1 << 24) - 256;
}

struct Kind {
  int n, m, threads;
  const void* fn;
};
template <class T, int kWN, int kWM, int kFN, int kFM, int kStages>
Kind kind_of() {
  typedef Tile<T, kWN, kWM, kFN, kFM, kStages> Own;
  return {Own::kN, Own::kM, Own::kThreads, reinterpret_cast<const void*>(&tiles_kernel<T, kWN, kWM, kFN, kFM, kStages>)};
}
template <class T>
Kind tile_kernel(int kind) {
  switch (kind) {
    case kFew: return {16, kFewTokens, 512, reinterpret_cast<const void*>(&few_kernel<T>)};
    case kBig: return {256, 256, 512, reinterpret_cast<const void*>(&big_tiles_kernel<T>)};
    case k64x128: return kind_of<T, 2, 2, 2, 1, 3>();
    case k128x64: return kind_of<T, 2, 2, 1, 2, 3>();
    default: return kind_of<T, 2, 2, 2, 2, 2>();
  }
}

rar_result_t project(const int8_t* const* xs, const int64_t* widths, const int64_t* x_strides, const float* x_scales,
                     const int8_t* const* weights, const int64_t* weight_strides, const float* weight_scales, int nranks, int64_t tokens,
                     int64_t outer, int dtype, const void* residual, int64_t residual_stride, void* const* recvbufs,
                     const int64_t* recv_strides, int nrecv, void* workspace, size_t workspace_bytes, void* stream) {
  int64_t total;
  if (rar_result_t r = check_widths(widths, nranks, &total)) return r;
  if (nrecv < 1 || nrecv > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "nrecv must be in [1, 64]");
  if (rar_result_t r = check_sizes(tokens, outer, dtype)) return r;
  if (tokens == 0) return RAR_SUCCESS;
  // so all tiles' threads are less than 2^32: 512 for 256 x 192 results at least,
  // or for what is left at the two edges
  if (tokens > kMaxResults / outer) return set_error(RAR_INVALID_ARGUMENT, "tokens * outer must be at most 2^38");
  if (!xs || !weights || !recvbufs) return set_error(RAR_INVALID_ARGUMENT, "an array of buffers is NULL");
  ProjArgs a{};
  const int64_t es = elem_size(dtype);
  std::vector<Block> reads, writes;
  reads.reserve(2 * nranks + 3);
  writes.reserve(nrecv + 1);
  for (int r = 0; r < nranks; ++r) {
    if (rar_result_t e = set_stride(a.x_stride[a.nranks], x_strides, r, widths[r], tokens, "input stride")) return e;
    int64_t w_stride;
    if (rar_result_t e = set_stride(w_stride, weight_strides, r, widths[r], outer, "weight stride")) return e;
    if (widths[r] == 0) continue;  // adds nothing
    if (rar_result_t e = check_pointer(xs[r], 1, "input", r)) return e;
    if (rar_result_t e = check_pointer(weights[r], 1, "weight", r)) return e;
    a.x[a.nranks] = xs[r];
    a.w[a.nranks] = weights[r];
    a.w_stride[a.nranks] = w_stride;
    a.width[a.nranks] = (int32_t)widths[r];
    reads.push_back({xs[r], tokens, widths[r], a.x_stride[a.nranks], "an input"});
    reads.push_back({weights[r], outer, widths[r], w_stride, "a weight"});
    ++a.nranks;
  }
  if (rar_result_t r = check_pointer(x_scales, 4, "x_scales")) return r;
  if (rar_result_t r = check_pointer(weight_scales, 4, "weight_scales")) return r;
  reads.push_back({x_scales, 1, tokens * 4, tokens * 4, "x_scales"});
  reads.push_back({weight_scales, 1, outer * 4, outer * 4, "weight_scales"});
  if (residual) {
    const int64_t given = residual_stride;
    if (rar_result_t e = set_stride(residual_stride, given ? &given : nullptr, 0, outer, tokens, "residual stride")) return e;
    if (rar_result_t e = check_pointer(residual, es, "residual")) return e;
    reads.push_back({residual, tokens, outer * es, residual_stride * es, "residual", kAnyOutput});
  }
  for (int k = 0; k < nrecv; ++k) {
    if (rar_result_t e = set_stride(a.dst_stride[k], recv_strides, k, outer, tokens, "output stride")) return e;
    if (rar_result_t e = check_pointer(recvbufs[k], es, "output", k)) return e;
    a.dst[k] = recvbufs[k];
    writes.push_back({recvbufs[k], tokens, outer * es, a.dst_stride[k] * es, "output"});
  }
  a.x_scales = x_scales;
  a.w_scales = weight_scales;
  a.residual = residual;
  a.residual_stride = residual_stride;
  a.tokens = tokens;
  a.outer = outer;
  a.ndst = nrecv;
  bool align_x = false, align_w = false;
  for (int r = 0; r < a.nranks; ++r) {
    a.steps += (a.width[r] + kDepth - 1) / kDepth;
    align_x = align_x || !is_aligned(a.x[r], a.x_stride[r], tokens);
    align_w = align_w || !is_aligned(a.w[r], a.w_stride[r], outer);
  }
  const Plan plan = plan_of(widths, nranks, tokens, outer, align_x, align_w);
  const int64_t need = plan.align_x + plan.align_w + plan.partial;
  if (need) {
    if (rar_result_t r = check_pointer(workspace, 1, "workspace")) return r;
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return set_error(RAR_INVALID_ARGUMENT, "workspace is not aligned to 16 bytes");
    if (workspace_bytes < (size_t)need) return set_error(RAR_INVALID_ARGUMENT, "workspace is too small");
    writes.push_back({workspace, 1, need, need, "workspace"});
  }
  if (rar_result_t r = check_blocks(reads, writes)) return r;
  const bool f32 = dtype == kFloat32;
  const Kind k = f32 ? tile_kernel<F32>(plan.kind) : tile_kernel<BF16>(plan.kind);
  a.tiles_m = (int32_t)((tokens + k.m - 1) / k.m);
  int64_t tiles_n = (outer + k.n - 1) / k.n, grid = 0;
  if (plan.kind == kBig) {
    // as many columns of 256 channels as make whole rounds of the CUs, the
    // rest in the size that leaves fewer of them idle
    const int64_t round = 256 / std::gcd<int64_t>(256, a.tiles_m), all = tiles_n;
    a.wide_n = (int32_t)(all / round * round);
    const int64_t rest = outer - a.wide_n * 256;
    auto cost = [&](int64_t width) { return (a.tiles_m * ((rest + width - 1) / width) + 255) / 256 * width; };
    if (rest > 0 && cost(192) >= cost(256)) a.wide_n = (int32_t)all;
    tiles_n = a.wide_n == all ? 0 : (rest + 191) / 192;
    grid = (a.tiles_m * (int64_t)a.wide_n + 7) / 8 * 8;
  }
  a.tiles_n = (int32_t)tiles_n;
  grid += (a.tiles_m * tiles_n + 7) / 8 * 8;
  if (plan.kind == kFew) grid = tiles_n;
  a.splits = plan.splits;
  char* work = static_cast<char*>(workspace);
  a.partial = reinterpret_cast<int32_t*>(work + plan.align_x + plan.align_w);
  AlignArgs aligned_x{}, aligned_w{};
  int64_t groups_x = 0, groups_w = 0;
  auto align = [&](AlignArgs& g, int64_t& groups, const int8_t** p, int64_t* stride, int64_t rows, char* to) -> rar_result_t {
    for (int r = 0; r < a.nranks; ++r) {
      const int64_t pitch = round_up(a.width[r], 16);
      g.src[r] = p[r], g.stride[r] = stride[r], g.dst[r] = reinterpret_cast<int8_t*>(to);
      g.width[r] = a.width[r];
      p[r] = reinterpret_cast<int8_t*>(to), stride[r] = pitch;
      to += rows * pitch;
      groups += (rows * (pitch / 16) + 255) / 256;
      if (groups > kMaxGroups) return set_error(RAR_INVALID_ARGUMENT, "tokens or outer times the widths is too large");
      g.first[r + 1] = (int32_t)groups;
    }
    g.rows = rows;
    g.nranks = a.nranks;
    return RAR_SUCCESS;
  };
  if (plan.align_x)
    if (rar_result_t r = align(aligned_x, groups_x, a.x, a.x_stride, tokens, work)) return r;
  if (plan.align_w)
    if (rar_result_t r = align(aligned_w, groups_w, a.w, a.w_stride, outer, work + plan.align_x)) return r;
  const void* align_fn = reinterpret_cast<const void*>(&align_kernel);
  if (rar_result_t r = launch_groups(align_fn, groups_x, 256, &aligned_x, &aligned_x.block0, stream)) return r;
  if (rar_result_t r = launch_groups(align_fn, groups_w, 256, &aligned_w, &aligned_w.block0, stream)) return r;
  if (rar_result_t r = launch_kernel(k.fn, dim3((unsigned)grid, (unsigned)a.splits), dim3(k.threads), &a, stream)) return r;
  if (a.splits == 1) return RAR_SUCCESS;
  const int vec = f32 ? F32::kVec : BF16::kVec;
  return launch_kernel(f32 ? reinterpret_cast<const void*>(&sum_kernel<F32>) : reinterpret_cast<const void*>(&sum_kernel<BF16>),
                       dim3((unsigned)((outer + 256 * vec - 1) / (256 * vec)), (unsigned)tokens), dim3(256), &a, stream);
}

}  // namespace
}  // namespace rar

extern "C" {

rar_result_t rar_quantize_rows(const void* const* xs, const int64_t* widths, const int64_t* x_strides, int nranks, int64_t rows,
                               rar_dtype_t dtype, int8_t* const* quantized, const int64_t* q_strides, float* scales, void* stream) {
  return rar::guarded([&] { return rar::quantize(xs, widths, x_strides, nranks, rows, dtype, quantized, q_strides, scales, stream); });
}

rar_result_t rar_int8_projection_allreduce(const int8_t* const* xs, const int64_t* widths, const int64_t* x_strides,
                                           const float* x_scales, const int8_t* const* weights, const int64_t* weight_strides,
                                           const float* weight_scales, int nranks, int64_t tokens, int64_t outer,
                                           rar_dtype_t dtype, const void* residual, int64_t residual_stride,
                                           void* const* recvbufs, const int64_t* recv_strides, int nrecv, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  return rar::guarded([&] {
    return rar::project(xs, widths, x_strides, x_scales, weights, weight_strides, weight_scales, nranks, tokens, outer, dtype, residual,
                        residual_stride, recvbufs, recv_strides, nrecv, workspace, workspace_bytes, stream);
  });
}

rar_result_t rar_int8_projection_workspace(const int64_t* widths, int nranks, int64_t tokens, int64_t outer, rar_dtype_t dtype,
                                           int aligned, size_t* bytes) {
  return rar::guarded([&]() -> rar_result_t {
    if (!bytes) return rar::set_error(RAR_INVALID_ARGUMENT, "bytes is NULL");
    int64_t total;
    if (rar_result_t r = rar::check_widths(widths, nranks, &total)) return r;
    if (rar_result_t r = rar::check_sizes(tokens, outer, dtype)) return r;
    const rar::Plan p = rar::plan_of(widths, nranks, tokens, outer, !aligned, !aligned);
    *bytes = tokens ? (size_t)(p.align_x + p.align_w + p.partial) : 0;
    return RAR_SUCCESS;
  });
}

}  // extern "C"
