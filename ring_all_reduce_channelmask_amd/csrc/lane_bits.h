// lane_bits.h -- 64-bit masks and a lane's own position in them, in 32-bit steps.
//
// No kernel shifts 64 bits by an amount that lanes hold: such a shift gave wrong
// results here where the amount was in the last vector register that the wave
// has, and where the compiler puts it is not for the source to say.  Amounts
// that are constants or the same for all lanes (in scalar registers) are fine.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace rar {

// How many of the mask's bits are below this lane's.
__device__ __forceinline__ int bits_below(uint64_t mask) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}
// Bit i (0 to 63) of the mask.  The empty assembly hides that the halves belong
// together: the compiler makes the choice of one a shift of 64 bits otherwise.
__device__ __forceinline__ bool bit_of(uint64_t mask, int i) {
  uint32_t low = (uint32_t)mask, high = (uint32_t)(mask >> 32);
  asm("" : "+v"(low), "+v"(high));
  return (i & 32 ? high : low) >> (i & 31) & 1;
}

}  // namespace rar
