// projection8.hip -- a row-parallel projection in 8-bit integers with its
// AllReduce, and the quantisation of rows split over the ranks.
//
//   quantise    a_t = max over r, k of |x_r[t,k]| / 127,   q_r[t,k] = rint(127 x_r[t,k] / max)
//   projection  y_c[t,d] = residual[t,d] + a_t b_d sum_r sum_k q_r[t,k] w_r[d,k]      c = every copy
//
// The scale of a token, and of a channel d of the weights, holds for all
// ranks: the sum over the ranks' columns is a sum of integers, exact, and the
// result does not depend on how the columns are split.
#include "op_common.h"

namespace rar {
namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxOuter = int64_t(1) << 24;
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
  int32_t nranks;
};

// rint(127 x / most), a tie to the even one as the quotient itself has it.
// bf16: 127 x is exact in fp32, and a quotient that is no tie is at least
// 2^-9 of itself away from one, far more than the division's rounding; both
// are scaled by a power of two where 127 x would leave fp32's range.  fp32:
// the same in 64 bits.
struct Quotient {
  float most, power;
  double most64;
  __device__ __forceinline__ explicit Quotient(float m) : most64(m) {
    power = m > 0x1p100f ? 0x1p-40f : m < 0x1p-60f ? 0x1p60f : 1.0f;
    most = m * power;
  }
  template <class T>
  __device__ __forceinline__ int32_t of(float x) const {
    if constexpr (T::kVec == 8) return (int32_t)__builtin_rintf(x * power * 127.0f / most);
    else return (int32_t)__builtin_rint((double)x * 127.0 / most64);
  }
};

// A workgroup takes a token: its columns of all ranks, in registers as far as
// kKept vectors a thread go, read a second time beyond that.
constexpr int kKept = 4;

template <class T>
__global__ void __launch_bounds__(256) quantize_kernel(QuantArgs) {
  const QuantArgs& args = kernel_args<QuantArgs>();
  __shared__ uint32_t scratch[4];
  const int64_t row = blockIdx.x;
  // vectors are counted through the ranks: each starts on a multiple of 256
  v4u kept[kKept];
  uint32_t most = 0;  // bits of |x|, which order as the values do, NaN last
  int n = 0;
  for (int r = 0; r < args.nranks; ++r) {
    const typename T::bits* p = static_cast<const typename T::bits*>(args.src[r]) + row * args.src_stride[r];
    for (int64_t e0 = 0; e0 < args.width[r]; e0 += 256 * T::kVec, ++n) {
      const int64_t e = e0 + threadIdx.x * T::kVec;
      v4u x = {0, 0, 0, 0};
      if (e < args.width[r]) x = load_part<T>(p + e, (int)(args.width[r] - e > T::kVec ? T::kVec : args.width[r] - e), 0);
#pragma unroll
      for (int j = 0; j < kKept; ++j)
        if (n == j) kept[j] = x;
      float f[T::kVec];
      T::widen(x, f);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) most = std::max(most, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) most = std::max(most, (uint32_t)__shfl_xor((int)most, d));
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) most = std::max(most, scratch[w]);
  const bool finite = most < 0x7F800000u;
  const float m = __uint_as_float(most);
  if (threadIdx.x == 0) args.scales[row] = finite ? m / 127.0f : __uint_as_float(0x7FC00000u);
  const bool zero = !finite || most == 0;
  const Quotient quotient(m);
  n = 0;
  for (int r = 0; r < args.nranks; ++r) {
    const typename T::bits* p = static_cast<const typename T::bits*>(args.src[r]) + row * args.src_stride[r];
    int8_t* out = args.dst[r] + row * args.dst_stride[r];
    for (int64_t e0 = 0; e0 < args.width[r]; e0 += 256 * T::kVec, ++n) {
      const int64_t e = e0 + threadIdx.x * T::kVec;
      if (e >= args.width[r]) continue;
      const int left = (int)(args.width[r] - e > T::kVec ? T::kVec : args.width[r] - e);
      v4u x = {0, 0, 0, 0};
      if (n < kKept) {
#pragma unroll
        for (int j = 0; j < kKept; ++j)
          if (n == j) x = kept[j];
      } else {
        x = load_part<T>(p + e, left, 0);
      }
      float f[T::kVec];
      T::widen(x, f);
      uint32_t q[T::kVec / 4];
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) {
        const uint32_t b = zero ? 0 : (uint32_t)quotient.of<T>(f[i]) & 0xFFu;
        q[i / 4] = i & 3 ? q[i / 4] | b << (8 * (i & 3)) : b;
      }
      if (left == T::kVec) {
        typedef uint32_t u32_user __attribute__((aligned(1)));
#pragma unroll
        for (int i = 0; i < T::kVec / 4; ++i) *reinterpret_cast<u32_user*>(out + e + 4 * i) = q[i];
      } else {
#pragma unroll
        for (int i = 0; i < T::kVec; ++i)
          if (i < left) out[e + i] = (int8_t)(q[i / 4] >> (8 * (i & 3)));
      }
    }
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
  int32_t nranks, ndst, tiles_m, tiles_n;
  int32_t steps;  // of kDepth bytes of the inner dimension, each rank's rounded up
};

// 16 bytes of a row from p on, n (1 or more) of them there and zeros behind.
// Fewer than 16 come as two overlapping pieces, neither beyond the n bytes.
__device__ __forceinline__ v4u load_bytes(const int8_t* p, int n) {
  typedef uint32_t v4u_byte __attribute__((ext_vector_type(4), aligned(1)));
  typedef uint64_t u64_byte __attribute__((aligned(1)));
  typedef uint32_t u32_byte __attribute__((aligned(1)));
  typedef uint16_t u16_byte __attribute__((aligned(1)));
  if (n >= 16) return *reinterpret_cast<const v4u_byte*>(p);
  uint64_t lo, hi = 0;
  if (n >= 8) {
    lo = *reinterpret_cast<const u64_byte*>(p);
    if (n > 8) hi = *reinterpret_cast<const u64_byte*>(p + n - 8) >> (8 * (16 - n));
  } else if (n >= 4) {
    const uint64_t end = *reinterpret_cast<const u32_byte*>(p + n - 4);
    lo = *reinterpret_cast<const u32_byte*>(p) | end << (8 * (n - 4));
  } else {
    lo = (uint8_t)p[0];
    if (n >= 2) lo |= (uint64_t)*reinterpret_cast<const u16_byte*>(p + n - 2) << (8 * (n - 2));
  }
  return v4u{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

constexpr int kTile = 128;   // tokens and channels of a workgroup
constexpr int kDepth = 128;  // bytes of the inner dimension at a time

template <class T>
__global__ void __launch_bounds__(256) tile_kernel(ProjArgs) {
  const ProjArgs& args = kernel_args<ProjArgs>();
  __shared__ __attribute__((aligned(16))) int8_t tile[2][kTile * kDepth];  // weights, tokens
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m0 = (int64_t)(blockIdx.x / args.tiles_n) * kTile, n0 = (int64_t)(blockIdx.x % args.tiles_n) * kTile;
  v16i acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0;
  for (int r = 0; r < args.nranks; ++r) {
    const int width = args.width[r];
    for (int k0 = 0; k0 < width; k0 += kDepth) {
      v4u a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = threadIdx.x + 256 * i, row = c >> 3, k = k0 + (c & 7) * 16;
        a[i] = b[i] = v4u{0, 0, 0, 0};
        if (k < width && n0 + row < args.outer) a[i] = load_bytes(args.w[r] + (n0 + row) * args.w_stride[r] + k, width - k);
        if (k < width && m0 + row < args.tokens) b[i] = load_bytes(args.x[r] + (m0 + row) * args.x_stride[r] + k, width - k);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = threadIdx.x + 256 * i, row = c >> 3, at = row * kDepth + (((c & 7) ^ (row >> 1 & 7)) << 4);
        *reinterpret_cast<v4u*>(&tile[0][at]) = a[i];
        *reinterpret_cast<v4u*>(&tile[1][at]) = b[i];
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        v4i wf[2], xf[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int wr = (wave & 1) * 64 + i * 32 + (lane & 31), xr = (wave >> 1) * 64 + i * 32 + (lane & 31), ch = s * 2 + (lane >> 5);
          wf[i] = *reinterpret_cast<const v4i*>(&tile[0][wr * kDepth + ((ch ^ (wr >> 1 & 7)) << 4)]);
          xf[i] = *reinterpret_cast<const v4i*>(&tile[1][xr * kDepth + ((ch ^ (xr >> 1 & 7)) << 4)]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[i], xf[j], acc[i][j], 0, 0, 0);
      }
    }
  }
  // lane l of a product has token l & 31 and channels 8 q + 4 (l >> 5) + 0..3
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t m = m0 + (wave >> 1) * 64 + j * 32 + (lane & 31);
    if (m >= args.tokens) continue;
    const float xs = args.x_scales[m];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = n0 + (wave & 1) * 64 + i * 32 + 8 * q + 4 * (lane >> 5);
        const int left = (int)(args.outer - n > 4 ? 4 : args.outer - n);
        if (left <= 0) continue;
        float f[4], ws[4];
        load4<F32>(reinterpret_cast<const uint32_t*>(args.w_scales + n), left, ws);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = (float)acc[i][j][4 * q + e] * xs * ws[e];
        if (args.residual) {
          float g[4];
          load4<T>(static_cast<const typename T::bits*>(args.residual) + m * args.residual_stride + n, left, g);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] += g[e];
        }
        for (int c = 0; c < args.ndst; ++c) store4<T>(static_cast<typename T::bits*>(args.dst[c]) + m * args.dst_stride[c] + n, left, f);
      }
    }
  }
}

// Many tokens: a tile of 256 tokens x 256 channels of a workgroup, whose
// operands go from memory to LDS without passing through registers, 128 bytes
// of the inner dimension at a time, while the step before is multiplied.
constexpr int kBig = 256;

// 16 bytes a lane from p to LDS, to 16 * lane behind `to`.  The caller waits
// for it (vmcnt) before a barrier.
__device__ __forceinline__ void to_lds(const int8_t* p, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(p) : "memory", "m0");
}

template <class T, int kWaves>
__global__ void __launch_bounds__(64 * kWaves, 1) big_tile_kernel(ProjArgs) {
  const ProjArgs& args = kernel_args<ProjArgs>();
  constexpr int kStage = 2 * kBig * kDepth;              // weights, then tokens
  constexpr int kWaveM = kBig * 2 / kWaves;              // tokens of a wave
  constexpr int kWaveN = 128;                            // channels of a wave
  constexpr int kFM = kWaveM / 32, kFN = kWaveN / 32;
  constexpr int kLoads = kBig * kDepth / 16 / (64 * kWaves);  // 16-byte loads a thread, of each operand
  __shared__ __attribute__((aligned(16))) int8_t lds[2 * kStage + 8192];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tile = (int64_t)(blockIdx.x & 7) * ((gridDim.x + 7) / 8) + (blockIdx.x >> 3);
  if (tile >= (int64_t)args.tiles_m * args.tiles_n) return;
  const int64_t m0 = tile % args.tiles_m * kBig, n0 = tile / args.tiles_m * kBig;
  v16i acc[kFN][kFM];
#pragma unroll
  for (int i = 0; i < kFN; ++i)
#pragma unroll
    for (int j = 0; j < kFM; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0;

  // the next step to load: rank, its inner offset, this lane's rows there
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t*)lds;
  const int row0 = wave * 8 + (lane >> 3), chunk = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));
  int rank = 0, k0 = 0;
  const int8_t *pw[kLoads], *px[kLoads];
  auto begin_rank = [&] {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int64_t row = row0 + i * 8 * kWaves;
      pw[i] = args.w[rank] + std::min(n0 + row, args.outer - 1) * args.w_stride[rank] + chunk * 16;
      px[i] = args.x[rank] + std::min(m0 + row, args.tokens - 1) * args.x_stride[rank] + chunk * 16;
    }
  };
  auto load_step = [&](int stage) {
    const int width = args.width[rank], left = width - k0;
    if (left >= kDepth) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        to_lds(pw[i] + k0, lds0 + stage * kStage + (i * kWaves + wave) * 1024);
        to_lds(px[i] + k0, lds0 + stage * kStage + kBig * kDepth + (i * kWaves + wave) * 1024);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        v4u a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
        if (left > chunk * 16) a = load_bytes(pw[i] + k0, left - chunk * 16), b = load_bytes(px[i] + k0, left - chunk * 16);
        *reinterpret_cast<v4u*>(&lds[stage * kStage + (i * kWaves + wave) * 1024 + lane * 16]) = a;
        *reinterpret_cast<v4u*>(&lds[stage * kStage + kBig * kDepth + (i * kWaves + wave) * 1024 + lane * 16]) = b;
      }
    }
    k0 += kDepth;
    if (k0 >= width && rank + 1 < args.nranks) {
      k0 = 0;
      ++rank;
      begin_rank();
    }
  };
  const int wn = (wave & 1) * kWaveN, wm = (wave >> 1) * kWaveM;
  if (args.steps > 0) {
    begin_rank();
    load_step(0);
  }
  for (int step = 0; step < args.steps; ++step) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    if (step + 1 < args.steps) load_step((step + 1) & 1);
    const int8_t* tw = &lds[(step & 1) * kStage];
    const int8_t* tx = tw + kBig * kDepth;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v4i wf[kFN], xf[kFM];
      // 32 rows apart the swizzle is the same
      const int r = lane & 31, at = r * kDepth + (((s * 2 + (lane >> 5)) ^ (r >> 1 & 7)) << 4);
#pragma unroll
      for (int i = 0; i < kFN; ++i) wf[i] = *reinterpret_cast<const v4i*>(&tw[(wn + i * 32) * kDepth + at]);
#pragma unroll
      for (int j = 0; j < kFM; ++j) xf[j] = *reinterpret_cast<const v4i*>(&tx[(wm + j * 32) * kDepth + at]);
#pragma unroll
      for (int i = 0; i < kFN; ++i)
#pragma unroll
        for (int j = 0; j < kFM; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[i], xf[j], acc[i][j], 0, 0, 0);
    }
  }
  // Out through LDS, 32 tokens x 128 channels of a wave at a time, so that
  // each row of it is read, completed and written as whole lines.
  constexpr int kPitch = kWaveN + 4;  // floats: rows start on different banks
  __syncthreads();
  float* own = reinterpret_cast<float*>(lds) + wave * 32 * kPitch;
  const int64_t n = n0 + wn + (lane & 15) * 8;
  const int left = (int)std::max<int64_t>(0, std::min<int64_t>(8, args.outer - n));
  float ws[8];
  load4<F32>(reinterpret_cast<const uint32_t*>(args.w_scales + n), left, ws);
  load4<F32>(reinterpret_cast<const uint32_t*>(args.w_scales + n + 4), left - 4, ws + 4);
#pragma unroll
  for (int j = 0; j < kFM; ++j) {
#pragma unroll
    for (int i = 0; i < kFN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v4f f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = (float)acc[i][j][4 * q + e];
        *reinterpret_cast<v4f*>(&own[(lane & 31) * kPitch + i * 32 + 8 * q + 4 * (lane >> 5)]) = f;
      }
    wave_lds_fence();
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int row = it * 4 + (lane >> 4);
      const int64_t m = m0 + wm + j * 32 + row;
      if (m >= args.tokens || left == 0) continue;
      const float xs = args.x_scales[m];
      float f[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v4f v = *reinterpret_cast<const v4f*>(&own[row * kPitch + (lane & 15) * 8 + 4 * h]);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * h + e] = v[e] * xs * ws[4 * h + e];
      }
      if (args.residual) {
        const typename T::bits* p = static_cast<const typename T::bits*>(args.residual) + m * args.residual_stride + n;
#pragma unroll
        for (int v = 0; v < 8 / T::kVec; ++v) {
          float g[T::kVec];
          T::widen(load_part<T>(p + v * T::kVec, std::max(0, left - v * T::kVec), 0), g);
#pragma unroll
          for (int e = 0; e < T::kVec; ++e) f[v * T::kVec + e] += g[e];
        }
      }
      for (int c = 0; c < args.ndst; ++c) {
        typename T::bits* p = static_cast<typename T::bits*>(args.dst[c]) + m * args.dst_stride[c] + n;
#pragma unroll
        for (int v = 0; v < 8 / T::kVec; ++v) store_part<T>(p + v * T::kVec, std::max(0, left - v * T::kVec), T::round(f + v * T::kVec));
      }
    }
    wave_lds_fence();
  }
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
  return launch_kernel(fn, dim3((unsigned)rows), dim3(256), &a, stream);
}

rar_result_t check_sizes(int64_t tokens, int64_t outer, int dtype) {
  if (rar_result_t r = check_float_dtype(dtype)) return r;
  if (tokens < 0 || tokens > kMaxTokens) return set_error(RAR_INVALID_ARGUMENT, "tokens must be in [0, 2^24]");
  if (outer < 1 || outer > kMaxOuter) return set_error(RAR_INVALID_ARGUMENT, "outer must be in [1, 2^24]");
  return RAR_SUCCESS;
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
  if (rar_result_t r = check_blocks(reads, writes)) return r;
  (void)workspace, (void)workspace_bytes;
  a.x_scales = x_scales;
  a.w_scales = weight_scales;
  a.residual = residual;
  a.residual_stride = residual_stride;
  a.tokens = tokens;
  a.outer = outer;
  a.ndst = nrecv;
  bool aligned = true;  // every row begins on a multiple of 16 bytes
  for (int r = 0; r < a.nranks; ++r) {
    a.steps += (a.width[r] + kDepth - 1) / kDepth;
    aligned = aligned && ((reinterpret_cast<uintptr_t>(a.x[r]) | reinterpret_cast<uintptr_t>(a.w[r]) | a.x_stride[r] | a.w_stride[r]) & 15) == 0;
  }
  const bool f32 = dtype == kFloat32;
  const bool big = aligned && tokens > 128;
  const int side = big ? kBig : kTile;
  const int64_t tiles_m = (tokens + side - 1) / side, tiles_n = (outer + side - 1) / side, tiles = tiles_m * tiles_n;
  if (tiles > 0x7FFFFFF0) return set_error(RAR_INVALID_ARGUMENT, "tokens * outer is too large");
  a.tiles_m = (int32_t)tiles_m;
  a.tiles_n = (int32_t)tiles_n;
  if (big) {
    constexpr int kWaves = 8;
    const void* fn = f32 ? reinterpret_cast<const void*>(&big_tile_kernel<F32, kWaves>) : reinterpret_cast<const void*>(&big_tile_kernel<BF16, kWaves>);
    return launch_kernel(fn, dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(64 * kWaves), &a, stream);
  }
  const void* fn = f32 ? reinterpret_cast<const void*>(&tile_kernel<F32>) : reinterpret_cast<const void*>(&tile_kernel<BF16>);
  return launch_kernel(fn, dim3((unsigned)tiles), dim3(256), &a, stream);
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
                                           size_t* bytes) {
  return rar::guarded([&]() -> rar_result_t {
    if (!bytes) return rar::set_error(RAR_INVALID_ARGUMENT, "bytes is NULL");
    int64_t total;
    if (rar_result_t r = rar::check_widths(widths, nranks, &total)) return r;
    if (rar_result_t r = rar::check_sizes(tokens, outer, dtype)) return r;
    *bytes = 0;
    return RAR_SUCCESS;
  });
}

}  // extern "C"
