// op_common.h -- what the operators around an AllReduce share (dropout.hip,
// logprobs.hip, adapters.hip): host-side argument checks, the C boundary's
// exception guard, and the device types and conversions.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <new>
#include <string>
#include <vector>

#include "capi_internal.h"

namespace rar {

// ---- host -------------------------------------------------------------------

// A rectangle of device memory that a call reads or writes: `rows` rows of
// `width` bytes, `stride` bytes apart.
constexpr int kNoOutput = -1, kAnyOutput = -2;
struct Block {
  const void* ptr;
  int64_t rows, width, stride;
  const char* what;
  int in_place = kNoOutput;  // of an input: the output (its place in the list) that may be exactly it
};

// Whether two rectangles share a byte.  Exact for equal strides (columns of
// one matrix are disjoint although their address ranges interleave);
// rectangles of different strides count as sharing where their ranges do.
inline bool blocks_overlap(const Block& a, const Block& b) {
  if (a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
  const int64_t pa = (int64_t)(uintptr_t)a.ptr, pb = (int64_t)(uintptr_t)b.ptr;
  const int64_t ea = pa + (a.rows - 1) * a.stride + a.width, eb = pb + (b.rows - 1) * b.stride + b.width;
  if (ea <= pb || eb <= pa) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  // A single row takes the other's stride: wider than that, it meets a row.
  const int64_t stride = a.rows > 1 ? a.stride : b.stride;
  if (a.rows > 1 && b.rows > 1 && a.stride != b.stride) return true;
  const int64_t d = (((pb - pa) % stride) + stride) % stride;  // b's column in a's rows
  return d < a.width || d + b.width > stride;
}

// Outputs share no byte with each other, and with an input only where both
// are the same rectangle and the input names that output: it may name one
// whose every element is written by the thread that reads the same element,
// after it has read it, and by no other.
inline rar_result_t check_blocks(const std::vector<Block>& reads, const std::vector<Block>& writes) {
  for (size_t i = 0; i < writes.size(); ++i) {
    for (size_t j = i + 1; j < writes.size(); ++j)
      if (blocks_overlap(writes[i], writes[j]))
        return set_error(RAR_INVALID_ARGUMENT, std::string(writes[i].what) + " " + std::to_string(i) + " overlaps " +
                                                   writes[j].what + " " + std::to_string(j));
    for (const Block& r : reads) {
      if (!blocks_overlap(writes[i], r)) continue;
      const bool same = writes[i].ptr == r.ptr && writes[i].rows == r.rows && writes[i].width == r.width &&
                        (writes[i].stride == r.stride || r.rows == 1);
      if (!same || (r.in_place != kAnyOutput && r.in_place != (int)i))
        return set_error(RAR_INVALID_ARGUMENT, std::string(writes[i].what) + " " + std::to_string(i) + " overlaps " + r.what);
    }
  }
  return RAR_SUCCESS;
}

inline rar_result_t check_float_dtype(int dtype) {
  if (dtype != RAR_FLOAT32 && dtype != RAR_BFLOAT16)
    return set_error(RAR_INVALID_ARGUMENT, "dtype must be float32 or bfloat16");
  return RAR_SUCCESS;
}

// `index` >= 0 names one of several; the message is made only on failure.
inline rar_result_t argument_error(const char* what, int index, const char* why) {
  return set_error(RAR_INVALID_ARGUMENT, what + (index < 0 ? std::string() : " " + std::to_string(index)) + " " + why);
}
// Rows `stride` elements apart, of `width` of them: the last row's offset is
// to stay below 2^60 bytes, beyond any memory and within 64-bit arithmetic.
// One row has no use for its stride, and gets its width.
inline rar_result_t set_stride(int64_t& stride, const int64_t* strides, int index, int64_t width, int64_t rows, const char* what) {
  stride = strides ? strides[index] : width;
  if (stride < width) return argument_error(what, index, "is below its width");
  if (rows <= 1) stride = width;
  else if (stride > (int64_t(1) << 58) / rows) return argument_error(what, index, "is out of range");
  return RAR_SUCCESS;
}
inline rar_result_t check_pointer(const void* p, size_t align, const char* what, int index = -1) {
  if (!p) return argument_error(what, index, "is NULL");
  if (reinterpret_cast<uintptr_t>(p) & (align - 1)) return argument_error(what, index, "is not aligned to its element size");
  return RAR_SUCCESS;
}

// Run the body of a C entry point: no C++ exception leaves it.
template <class F>
rar_result_t guarded(F&& body) {
  try {
    clear_error();
    return body();
  } catch (...) {
    try {
      return set_error(RAR_INTERNAL_ERROR, "out of host memory");
    } catch (...) {
      return RAR_INTERNAL_ERROR;
    }
  }
}

inline rar_result_t launch_kernel(const void* fn, dim3 grid, dim3 block, void* args, void* stream) {
  void* params[] = {args};
  const hipError_t e = hipLaunchKernel(fn, grid, block, params, 0, reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return set_error(RAR_HIP_ERROR, std::string("kernel launch failed: ") + hipGetErrorString(e));
  return RAR_SUCCESS;
}

// ---- device -----------------------------------------------------------------

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
// Rows and buffers need only element alignment: gfx950 serves unaligned
// global vector accesses in hardware.
typedef uint32_t v4u_user __attribute__((ext_vector_type(4), aligned(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v4u load_nt(const void* p) {
  return __builtin_nontemporal_load(static_cast<const v4u_user*>(p));
}
__device__ __forceinline__ v4u load_16(const void* p) { return *static_cast<const v4u_user*>(p); }
__device__ __forceinline__ void store_nt(void* p, v4u v) {
  __builtin_nontemporal_store((v4u_user)v, static_cast<v4u_user*>(p));
}

// Payload types: how many elements a 16-byte vector holds, widening to fp32
// (exact) and rounding to nearest even.
struct F32 {
  typedef uint32_t bits;
  static constexpr int kVec = 4;
  static constexpr uint32_t kNegInf = 0xFF800000u;  // a word of -inf elements
  static __device__ __forceinline__ void widen(v4u x, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(x[i]);
  }
  static __device__ __forceinline__ v4u round(const float* f) {
    v4u r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(f[i]);
    return r;
  }
  static __device__ __forceinline__ float widen1(bits x) { return __uint_as_float(x); }
  static __device__ __forceinline__ bits round1(float f) { return __float_as_uint(f); }
};
struct BF16 {
  typedef uint16_t bits;
  static constexpr int kVec = 8;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  static __device__ __forceinline__ void widen(v4u x, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(x[i] << 16);
      f[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ v4u round(const float* f) {
    v4u r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{f[2 * i], f[2 * i + 1]}, v2bf));
    return r;
  }
  static __device__ __forceinline__ float widen1(bits x) { return __uint_as_float((uint32_t)x << 16); }
  static __device__ __forceinline__ bits round1(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};

// A kernel's arguments (its only parameter, of type A) where the launch put
// them.  Through the parameter itself a large structure that is indexed at run
// time may be copied to scratch memory first.
template <class A>
__device__ __forceinline__ const A& kernel_args() {
  typedef const __attribute__((address_space(4))) A* P;
  return *(const A*)(P)__builtin_amdgcn_kernarg_segment_ptr();
}

// The first `n` (0..kVec) elements at p as a vector, the rest -inf or zero.
template <class T>
__device__ __forceinline__ v4u load_part(const typename T::bits* p, int n, uint32_t fill) {
  if (n >= T::kVec) return load_nt(p);
  v4u r = {fill, fill, fill, fill};
#pragma unroll
  for (int i = 0; i < T::kVec; ++i) {
    if (i < n) {
      if constexpr (T::kVec == 4) {
        r[i] = p[i];
      } else {
        const int sh = 16 * (i & 1);
        r[i / 2] = (r[i / 2] & ~(0xFFFFu << sh)) | ((uint32_t)p[i] << sh);
      }
    }
  }
  return r;
}
template <class T>
__device__ __forceinline__ void store_part(typename T::bits* p, int n, v4u v) {
  if (n >= T::kVec) {
    store_nt(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < T::kVec; ++i) {
    if (i < n) {
      if constexpr (T::kVec == 4) p[i] = v[i];
      else p[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
  }
}

// Combine each lane's value over its group of n = 1, 2, 4 ... 32 lanes, with
// lane moves inside the vector unit up to 16.
template <int n, class Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
#define RAR_STEP(ctrl) \
  v = op(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, 0xF, 0xF, true)))
  if constexpr (n > 1) RAR_STEP(0xB1);   // lane ^ 1
  if constexpr (n > 2) RAR_STEP(0x4E);   // lane ^ 2
  if constexpr (n > 4) RAR_STEP(0x141);  // mirrored within 8
  if constexpr (n > 8) RAR_STEP(0x140);  // mirrored within 16
#undef RAR_STEP
  if constexpr (n > 16) v = op(v, __shfl_xor(v, 16));
  return v;
}

// Between a wave's stores to LDS and its own loads: LDS keeps a wave's order,
// so only the compiler has to.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A vector without its first n (0 or more) elements, zeros behind.
template <class T>
__device__ __forceinline__ v4u shift_elements(v4u v, int n) {
  const int bits = n * (128 / T::kVec);
  uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
  if (bits >= 64) lo = hi, hi = 0;
  const int b = bits & 63;
  lo = b ? lo >> b | hi << (64 - b) : lo;
  hi >>= b;
  return bits >= 128 ? v4u{0, 0, 0, 0} : v4u{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Four neighbouring elements, `n` of them there, as fp32.
template <class T>
__device__ __forceinline__ void load4(const typename T::bits* p, int n, float* f) {
  typedef uint32_t v2u_user __attribute__((ext_vector_type(2), aligned(2)));
  if (n >= 4) {
    if constexpr (T::kVec == 4) {
      T::widen(load_16(p), f);
    } else {
      const v2u v = *reinterpret_cast<const v2u_user*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = T::widen1((uint16_t)(v[i / 2] >> (16 * (i & 1))));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = 0.0f;
      if (i < n) f[i] = T::widen1(p[i]);
    }
  }
}
template <class T>
__device__ __forceinline__ void store4(typename T::bits* p, int n, const float* f) {
  typedef uint32_t v2u_user __attribute__((ext_vector_type(2), aligned(2)));
  if (n >= 4) {
    if constexpr (T::kVec == 4) {
      *reinterpret_cast<v4u_user*>(p) = T::round(f);
    } else {
      v2u v;
#pragma unroll
      for (int i = 0; i < 2; ++i) v[i] = (uint32_t)T::round1(f[2 * i]) | (uint32_t)T::round1(f[2 * i + 1]) << 16;
      *reinterpret_cast<v2u_user*>(p) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = T::round1(f[i]);
  }
}

}  // namespace rar
