// fp32 -> bf16, for every kernel: the hardware conversion, one instruction for two values.
// Round to nearest even, subnormals kept; a NaN stays a NaN whichever of its bits are set
// (rounded as an integer, one with its low bits set would carry into the sign and leave a
// zero).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {
namespace {

// lo in the low half
__device__ __forceinline__ uint32_t bf16x2_rne(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
__device__ __forceinline__ uint16_t bf16_rne(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

}  // namespace
}  // namespace fp8q
