// dropout.hip -- the one-shot AllReduce with dropout and a residual in its
// epilogue, and its gradient; the dropout mask is never stored.
//
//   forward   y_k[i] = residual[i] + drop(sum_r x_r[i])        k = every copy
//   gradient  dresidual[i] = sum_k dy_k[i],  dx_r[i] = drop(dresidual[i])
//   drop(v) at i = v * 65536 / (65536 - cut) if field(i) >= cut, else 0
//
// field(i) is 16 of the 128 bits that Philox4x32 with 7 rounds (Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011:
// the fewest rounds that pass its statistical tests) gives for the key
// `seed` and the counter (i / 8, offset): one evaluation serves 8 elements,
// and the gradient evaluates it again instead of reading a mask.  Sums are
// fp32 in rank order and everything is rounded to the payload type once.
//
// Bound by memory: (inputs + residual + outputs) * count elements move once.
// Seven rounds cost 14 products of 32 x 32 bits for 8 elements, which hides
// behind the loads.  Measured (kernel): 4 ranks of 16M fp32 with a residual
// 100 us = 6.0 TB/s; 8 ranks of 32M bf16, gradient, 195 us = 5.5 TB/s (189 to
// 198 on other machines); 4 ranks of 104 x 7168 bf16 5.5 us; 7168 elements 3.3
// us.
#include "op_common.h"

#include <cmath>

namespace rar {
namespace {

struct DropoutArgs {
  const void* src[kMaxRanks];
  void* dst[kMaxRanks];
  const void* residual;  // forward: added after the dropout, or NULL
  void* dresidual;       // gradient: the undropped sum, or NULL
  const uint64_t* rng;   // {seed, offset} in device memory
  uint64_t call;         // added to the offset
  int64_t count;
  int32_t nsrc, ndst;
  uint32_t cut;          // of 65536: a field below it drops the element
  float factor;          // 65536 / (65536 - cut)
};

// The 8 fields of elements 8n .. 8n+7, two to a word, the lower element in
// the lower half.
__device__ __forceinline__ v4u philox7(uint64_t n, uint64_t seed, uint64_t offset) {
  uint32_t a = (uint32_t)n, b = (uint32_t)(n >> 32), c = (uint32_t)offset, d = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int round = 0; round < 7; ++round) {
    const uint64_t u = (uint64_t)a * 0xD2511F53u, v = (uint64_t)c * 0xCD9E8D57u;
    a = (uint32_t)(v >> 32) ^ b ^ k0;
    b = (uint32_t)v;
    c = (uint32_t)(u >> 32) ^ d ^ k1;
    d = (uint32_t)u;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return v4u{a, b, c, d};
}

// A wave takes 64 generator calls, 512 elements, at a time.  In bf16 a lane
// has one 16-byte vector, the 8 elements of its own call.  In fp32 it has two,
// 64 vectors apart, so that each load and store of the wave covers whole
// lines (with neighbouring vectors, each store would cover half of every
// line it touches: 16M x 4 ranks 161 us, this way 104 us); vector v needs
// half v % 2 of call v / 2, which another lane drew.
template <class T>
struct Fields;
template <>
struct Fields<BF16> {
  static __device__ __forceinline__ void get(v4u mine, int, uint32_t* field) {
#pragma unroll
    for (int j = 0; j < 8; ++j) field[j] = j & 1 ? mine[j / 2] >> 16 : mine[j / 2] & 0xFFFFu;
  }
};
template <>
struct Fields<F32> {
  static __device__ __forceinline__ void get(v4u mine, int lane, uint32_t* field) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int from = (v * 32 + lane / 2) * 4;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t even = __builtin_amdgcn_ds_bpermute(from, (int)mine[w]);
        const uint32_t odd = __builtin_amdgcn_ds_bpermute(from, (int)mine[w + 2]);
        const uint32_t word = lane & 1 ? odd : even;
        field[v * 4 + w * 2] = word & 0xFFFFu;
        field[v * 4 + w * 2 + 1] = word >> 16;
      }
    }
  }
};

// This lane's vectors of the wave's 512 elements from `base`; `left` elements
// are there from `base` on.
template <class T>
struct Group {
  static constexpr int kVecs = 8 / T::kVec;
  v4u v[kVecs];
  __device__ __forceinline__ void load(const void* buf, int64_t base, int64_t left, int lane, bool full) {
    const typename T::bits* p = static_cast<const typename T::bits*>(buf) + base;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int e = (j * 64 + lane) * T::kVec;
      v[j] = full ? load_nt(p + e) : load_part<T>(p + e, left - e > 8 ? 8 : (int)(left - e), 0);
    }
  }
  __device__ __forceinline__ void widen(float* f) const {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) T::widen(v[j], f + j * T::kVec);
  }
  static __device__ __forceinline__ void store(void* buf, int64_t base, int64_t left, int lane, bool full, const float* f) {
    typename T::bits* p = static_cast<typename T::bits*>(buf) + base;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int e = (j * 64 + lane) * T::kVec;
      const v4u o = T::round(f + j * T::kVec);
      if (full) store_nt(p + e, o);
      else store_part<T>(p + e, left - e > 8 ? 8 : (int)(left - e), o);
    }
  }
};

template <class T, bool kBackward>
__global__ void __launch_bounds__(256) dropout_kernel(DropoutArgs) {
  const DropoutArgs& args = kernel_args<DropoutArgs>();
  constexpr int kBatch = 4;  // inputs whose loads are issued together
  const uint64_t seed = args.rng[0], offset = args.rng[1] + args.call;
  const int lane = threadIdx.x & 63;
  const int64_t waves = (args.count + 511) / 512;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < waves; i += (int64_t)gridDim.x * 4) {
    const int64_t base = i * 512, left = args.count - base;
    const bool full = left >= 512;
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    for (int r0 = 0; r0 < args.nsrc; r0 += kBatch) {
      Group<T> x[kBatch];
#pragma unroll
      for (int r = 0; r < kBatch; ++r)
        if (r0 + r < args.nsrc) x[r].load(args.src[r0 + r], base, left, lane, full);
#pragma unroll
      for (int r = 0; r < kBatch; ++r) {
        if (r0 + r < args.nsrc) {
          float f[8];
          x[r].widen(f);
#pragma unroll
          for (int j = 0; j < 8; ++j) sum[j] = r0 + r == 0 ? f[j] : sum[j] + f[j];
        }
      }
    }
    uint32_t field[8];
    Fields<T>::get(philox7((uint64_t)(i * 64 + lane), seed, offset), lane, field);
    float out[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = field[j] >= args.cut ? sum[j] * args.factor : 0.0f;
    if (kBackward) {
      if (args.dresidual) Group<T>::store(args.dresidual, base, left, lane, full, sum);
    } else if (args.residual) {
      Group<T> res;
      res.load(args.residual, base, left, lane, full);
      float f[8];
      res.widen(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] += f[j];
    }
    for (int k = 0; k < args.ndst; ++k) Group<T>::store(args.dst[k], base, left, lane, full, out);
  }
}

const void* get_dropout_kernel(int dtype, bool backward) {
  if (dtype == kFloat32)
    return backward ? reinterpret_cast<const void*>(&dropout_kernel<F32, true>)
                    : reinterpret_cast<const void*>(&dropout_kernel<F32, false>);
  return backward ? reinterpret_cast<const void*>(&dropout_kernel<BF16, true>)
                  : reinterpret_cast<const void*>(&dropout_kernel<BF16, false>);
}

rar_result_t dropout_call(const void* const* src, int nsrc, void* const* dst, int ndst, const void* residual,
                          void* dresidual, size_t count, int dtype, double p, const void* rng, uint64_t call,
                          void* stream, bool backward) {
  if (nsrc < 1 || nsrc > kMaxRanks || ndst < 1 || ndst > kMaxRanks)
    return set_error(RAR_INVALID_ARGUMENT, "the numbers of inputs and outputs must be in [1, 64]");
  if (rar_result_t r = check_float_dtype(dtype)) return r;
  if (!(p >= 0.0 && p <= 1.0)) return set_error(RAR_INVALID_ARGUMENT, "p must be in [0, 1]");
  if (count == 0) return RAR_SUCCESS;
  if (count > (size_t(1) << 40)) return set_error(RAR_INVALID_ARGUMENT, "count too large");
  if (!src || !dst) return set_error(RAR_INVALID_ARGUMENT, "an array of buffers is NULL");
  const size_t es = (size_t)elem_size(dtype);
  if (rar_result_t r = check_pointer(rng, 8, "rng")) return r;
  DropoutArgs a{};
  const int64_t bytes = (int64_t)(count * es);
  // A thread reads and writes the same elements of all buffers.
  std::vector<Block> reads, writes;
  reads.reserve(nsrc + 2);
  writes.reserve(ndst + 1);
  reads.push_back({rng, 1, 16, 16, "rng"});
  for (int r = 0; r < nsrc; ++r) {
    if (rar_result_t e = check_pointer(src[r], es, "input", r)) return e;
    a.src[r] = src[r];
    reads.push_back({src[r], 1, bytes, bytes, "an input", kAnyOutput});
  }
  for (int k = 0; k < ndst; ++k) {
    if (rar_result_t e = check_pointer(dst[k], es, "output", k)) return e;
    a.dst[k] = dst[k];
    writes.push_back({dst[k], 1, bytes, bytes, "output"});
  }
  if (residual) {
    if (rar_result_t e = check_pointer(residual, es, "residual")) return e;
    reads.push_back({residual, 1, bytes, bytes, "residual", kAnyOutput});
  }
  if (dresidual) {
    if (rar_result_t e = check_pointer(dresidual, es, "dresidual")) return e;
    writes.push_back({dresidual, 1, bytes, bytes, "dresidual"});
  }
  if (rar_result_t r = check_blocks(reads, writes)) return r;
  a.residual = residual;
  a.dresidual = dresidual;
  a.rng = static_cast<const uint64_t*>(rng);
  a.call = call;
  a.count = (int64_t)count;
  a.nsrc = nsrc;
  a.ndst = ndst;
  a.cut = (uint32_t)std::nearbyint(p * 65536.0);
  a.factor = a.cut < 65536u ? (float)(65536.0 / (65536.0 - a.cut)) : 0.0f;
  // One pass of a wave each: a new workgroup's loads start while others store
  // (8 ranks of 32M bf16, on one machine: 2048 workgroups 206 us, 4096 198, 8192
  // 192, all 190).
  const int64_t blocks = std::min<int64_t>(((int64_t)count + 2047) / 2048, 65536);
  return launch_kernel(get_dropout_kernel(dtype, backward), dim3((unsigned)blocks), dim3(256), &a, stream);
}

}  // namespace
}  // namespace rar

extern "C" {

rar_result_t rar_dropout_allreduce(const void* const* sendbufs, int nsend, void* const* recvbufs, int nrecv,
                                   const void* residual, size_t count, rar_dtype_t dtype, double p,
                                   const void* rng, uint64_t call, void* stream) {
  return rar::guarded([&] {
    return rar::dropout_call(sendbufs, nsend, recvbufs, nrecv, residual, nullptr, count, dtype, p, rng, call, stream,
                             false);
  });
}

rar_result_t rar_dropout_allreduce_backward(const void* const* grads, int ngrads, void* const* dsends, int ndsends,
                                            void* dresidual, size_t count, rar_dtype_t dtype, double p,
                                            const void* rng, uint64_t call, void* stream) {
  return rar::guarded([&] {
    return rar::dropout_call(grads, ngrads, dsends, ndsends, nullptr, dresidual, count, dtype, p, rng, call, stream,
                             true);
  });
}

}  // extern "C"
