// Reductions over a wave of 64 lanes, and router logits (routing, norm and balance
// kernels).
#pragma once

#include "quant_common.h"

namespace fp8q {
namespace {

// maximum over the wave, uniform
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = dpp_row_max_u32(v);
  const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16));
  const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48));
  return max(a, b);
}

// sum over the wave, uniform: as the maximum, within 16-lane rows by DPP, the
// rows in order
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float lane_f32(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ float wave_sum_f32(float v) {
  v += dpp_f32<0xB1>(v);
  v += dpp_f32<0x4E>(v);
  v += dpp_f32<0x141>(v);
  v += dpp_f32<0x140>(v);
  return (lane_f32(v, 0) + lane_f32(v, 16)) + (lane_f32(v, 32) + lane_f32(v, 48));
}

// e^x, x <= 0 (2 ulp; below e^-87 the result may be flushed to zero)
__device__ __forceinline__ float exp_neg(float x) { return exp_f32(fmaxf(x, -110.0f)); }

// Finite logits as unsigned keys in the same order, all above kNoKey; -inf and
// NaN are kNoKey (never chosen), +inf counts as the largest finite value.
constexpr uint32_t kNoKey = 0;
__device__ __forceinline__ float clean_logit(float l) {
  return l == l ? fminf(l, 3.402823466e38f) + 0.0f : -INFINITY;  // + 0: -0 ties with +0
}
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t u = __float_as_uint(l);
  return l == -INFINITY ? kNoKey : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

}  // namespace
}  // namespace fp8q
