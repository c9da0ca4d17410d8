// Balance loss of a top-k router, and the gradient of its logits, on gfx950.
//
//   p[t]     = softmax(logits[t]) over the experts that can be chosen (-inf and NaN
//              cannot; +inf counts as the largest finite value, as in the routing)
//   n        = tokens with such an expert;  counts[e] = slots of expert e
//   prob[e]  = sum_t p[t][e] / n,   f[e] = counts[e] / (n * top_k)
//   loss     = coef * E * sum_e f[e] * prob[e]
//
// Gradient, f being constant: with c[e] = coef * E * f[e] / n * dloss
//   dl[e] = p[e] * (c[e] - sum_i p[i] c[i])
// and through the weights of the chosen slots j (ids e_j, gradients dw_j), w being
// p or, renormalised, the softmax over the chosen slots alone, m[e] slots holding e:
//   dl[e] += w[e] * (sum_{j: e_j = e} dw_j - (m[e] or 1) * sum_j w[e_j] dw_j)
//
// A wave takes its tokens one after the other, lane l holding the logits l, l + 64,
// ...  Probabilities are summed in registers, then over a workgroup's waves and over
// the workgroups in a fixed order; counts are integers, so their LDS atomics give
// the same result in any order.
#include <algorithm>

#include "wave_common.h"

namespace fp8q {
namespace {

constexpr uint32_t kWaves = 16, kThreads = 64 * kWaves;
// One workgroup takes up to this many tokens alone (one launch); beyond, at least
// kBlockTokens a workgroup and at most kMaxBlocks of them, summed by a second one.
constexpr uint32_t kLoneTokens = 128, kBlockTokens = 32, kMaxBlocks = 128;

uint32_t balance_blocks(uint32_t T) {
  return T <= kLoneTokens ? 1 : std::min((T + kBlockTokens - 1) / kBlockTokens, kMaxBlocks);
}

// This lane's logits of token t as fp32; -inf where there is none or NaN.
template <int NV>
__device__ __forceinline__ void load_logits(const void* logits, bool bf16, uint32_t t, uint32_t E, uint32_t lane,
                                            float (&l)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t e = 64 * i + lane;
    const uint64_t at = (uint64_t)t * E + min(e, E - 1);
    const float v = bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[at] << 16)
                         : static_cast<const float*>(logits)[at];
    l[i] = e < E ? clean_logit(v) : -INFINITY;
  }
}

// The key of the largest logit.
template <int NV>
__device__ __forceinline__ uint32_t top_key(const float (&l)[NV]) {
  uint32_t top = kNoKey;
#pragma unroll
  for (int i = 0; i < NV; ++i) top = max(top, logit_key(l[i]));
  return wave_max_u32(top);
}

// e[i] = e^(l[i] - top), 0 where l is -inf; returns their sum (0: nothing to choose).
template <int NV>
__device__ __forceinline__ float exp_logits(const float (&l)[NV], uint32_t top, float (&e)[NV]) {
  const float lmax = top == kNoKey ? 0.0f : key_logit(top);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    e[i] = l[i] == -INFINITY ? 0.0f : exp_neg(l[i] - lmax);
    sum += e[i];
  }
  return wave_sum_f32(sum);
}

struct BalanceArgs {
  const void* logits;
  const int32_t* ids;
  int32_t* counts;  // [E + 1], the last one n
  float *prob, *loss;
  uint32_t* part;  // [blocks][2][E + 1]: probability sums, counts; unused by a lone workgroup
  float coef;
  uint32_t T, E, k, blocks;
  bool bf16;
};

// counts, prob and the loss from the sums in psum[E] and cnt[E + 1] (LDS).
// Called by the whole workgroup.
__device__ __forceinline__ void finish(const BalanceArgs& a, const float* psum, const uint32_t* cnt, float* red) {
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t n = cnt[a.E];
  const float rn = n ? (float)n : 1.0f;
  float dot = 0.0f;
  for (uint32_t e = threadIdx.x; e < a.E; e += kThreads) {
    const float p = psum[e] / rn;
    a.prob[e] = p;
    a.counts[e] = (int32_t)cnt[e];
    dot += (float)cnt[e] / (rn * (float)a.k) * p;
  }
  if (threadIdx.x == 0) a.counts[a.E] = (int32_t)n;
  dot = wave_sum_f32(dot);
  if (lane == 0) red[wave] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (uint32_t w = 0; w < kWaves; ++w) s += red[w];
    *a.loss = a.coef * (float)a.E * s;
  }
}

template <int NV>
__global__ __launch_bounds__(kThreads) void balance_kernel(BalanceArgs a) {
  extern __shared__ uint32_t lds[];  // [E + 1] counts, [kWaves][E] probabilities
  __shared__ float red[kWaves];
  uint32_t* cnt = lds;
  float* sums = reinterpret_cast<float*>(lds + a.E + 1);
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (uint32_t e = threadIdx.x; e <= a.E; e += kThreads) cnt[e] = 0;
  __syncthreads();
  float acc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.0f;
  uint32_t n = 0;
  for (uint32_t t = blockIdx.x * kWaves + wave; t < a.T; t += gridDim.x * kWaves) {
    float l[NV], x[NV];
    load_logits<NV>(a.logits, a.bf16, t, a.E, lane, l);
    const uint32_t id = lane < a.k ? (uint32_t)a.ids[(uint64_t)t * a.k + lane] : a.E;
    const float sum = exp_logits<NV>(l, top_key<NV>(l), x);
    if (sum > 0.0f) {  // uniform
      const float r = 1.0f / sum;
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] = __builtin_fmaf(x[i], r, acc[i]);
      ++n;
    }
    if (id < a.E) atomicAdd(&cnt[id], 1u);
  }
  if (lane == 0 && n) atomicAdd(&cnt[a.E], n);
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (64 * i + lane < a.E) sums[wave * a.E + 64 * i + lane] = acc[i];
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < a.E; e += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) s += sums[w * a.E + e];
    sums[e] = s;
  }
  __syncthreads();
  if (a.blocks == 1) {
    finish(a, sums, cnt, red);
  } else {
    uint32_t* out = a.part + (uint64_t)blockIdx.x * 2 * (a.E + 1);
    for (uint32_t e = threadIdx.x; e <= a.E; e += kThreads) {
      if (e < a.E) out[e] = __float_as_uint(sums[e]);
      out[a.E + 1 + e] = cnt[e];
    }
  }
}

// The workgroups' sums, added in order.
__global__ __launch_bounds__(kThreads) void balance_sum_kernel(BalanceArgs a) {
  extern __shared__ uint32_t lds[];  // [E + 1] counts, [slices][E + 1] twice
  __shared__ float red[kWaves];
  const uint32_t EB = a.E + 1, slices = kThreads / EB ? kThreads / EB : 1;
  uint32_t* cnt = lds;
  float* psum = reinterpret_cast<float*>(lds + EB);
  uint32_t* csum = lds + EB + slices * EB;
  const uint32_t slice = threadIdx.x / EB, e = threadIdx.x % EB;
  if (slice < slices) {
    float p = 0.0f;
    uint32_t c = 0;
    for (uint32_t b = slice; b < a.blocks; b += slices) {
      const uint32_t* in = a.part + (uint64_t)b * 2 * EB;
      if (e < a.E) p += __uint_as_float(in[e]);
      c += in[EB + e];
    }
    psum[slice * EB + e] = p;
    csum[slice * EB + e] = c;
  }
  __syncthreads();
  if (threadIdx.x < EB) {
    float p = 0.0f;
    uint32_t c = 0;
    for (uint32_t s = 0; s < slices; ++s) {
      p += psum[s * EB + threadIdx.x];
      c += csum[s * EB + threadIdx.x];
    }
    psum[threadIdx.x] = p;
    cnt[threadIdx.x] = c;
  }
  __syncthreads();
  finish(a, psum, cnt, red);
}

struct RouteGradArgs {
  const void* logits;
  const int32_t* ids;       // NULL: no weights' gradient
  const float* dweights;
  const int32_t* counts;    // NULL: no balance loss
  const float* dloss;       // NULL: 1
  void* dlogits;
  float coef;
  uint32_t T, E, k;
  bool bf16, renorm;
};

template <int NV>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs a) {
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float share[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) share[i] = 0.0f;
  if (a.counts) {
    const float n = (float)a.counts[a.E];
    if (n > 0.0f) {
      const float f = a.coef * (float)a.E / (n * (float)a.k) / n * (a.dloss ? *a.dloss : 1.0f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (64 * i + lane < a.E) share[i] = f * (float)a.counts[64 * i + lane];
    }
  }
  for (uint32_t t = blockIdx.x * 4 + wave; t < a.T; t += gridDim.x * 4) {
    float l[NV], x[NV], g[NV];
    load_logits<NV>(a.logits, a.bf16, t, a.E, lane, l);
    const bool slot = a.ids && lane < a.k;
    const uint32_t id = slot ? (uint32_t)a.ids[(uint64_t)t * a.k + lane] : a.E;
    const float dwj = id < a.E ? a.dweights[(uint64_t)t * a.k + lane] : 0.0f;
    const uint32_t top = top_key<NV>(l);
    const float sum = exp_logits<NV>(l, top, x);
    const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) dot = __builtin_fmaf(x[i] * r, share[i], dot);
    dot = wave_sum_f32(dot);
#pragma unroll
    for (int i = 0; i < NV; ++i) g[i] = x[i] * r * (share[i] - dot);
    if (a.ids) {
      float d[NV], m[NV];  // the slots' gradients and number at this lane's experts
#pragma unroll
      for (int i = 0; i < NV; ++i) d[i] = m[i] = 0.0f;
      for (uint32_t j = 0; j < a.k; ++j) {
        const uint32_t ej = (uint32_t)__builtin_amdgcn_readlane((int)id, (int)j);
        const float dj = lane_f32(dwj, (int)j);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (ej == 64 * i + lane) {
            d[i] += dj;
            m[i] += 1.0f;
          }
      }
      float rw = r;
      if (a.renorm) {
        // over the chosen slots alone, with their own maximum: chosen by another
        // rule than the largest logits, they may all lie far below the top
        float c[NV], mass = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] = m[i] > 0.0f ? l[i] : -INFINITY;
        const uint32_t top_c = top_key<NV>(c);
        if (top_c != top) exp_logits<NV>(c, top_c, x);  // uniform
#pragma unroll
        for (int i = 0; i < NV; ++i) mass = __builtin_fmaf(x[i], m[i], mass);
        mass = wave_sum_f32(mass);
        rw = mass > 0.0f ? 1.0f / mass : 0.0f;
      }
      float wd = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) wd = __builtin_fmaf(x[i] * rw, d[i], wd);
      wd = wave_sum_f32(wd);
#pragma unroll
      for (int i = 0; i < NV; ++i) g[i] += x[i] * rw * (d[i] - (a.renorm ? m[i] : 1.0f) * wd);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t e = 64 * i + lane;
      if (e < a.E) {
        const uint64_t at = (uint64_t)t * a.E + e;
        if (a.bf16)
          static_cast<uint16_t*>(a.dlogits)[at] = (uint16_t)bf16_bits_rne(g[i]);
        else
          static_cast<float*>(a.dlogits)[at] = g[i];
      }
    }
  }
}

template <int NV>
hipError_t launch_balance_nv(const BalanceArgs& a, hipStream_t s) {
  const size_t lds = (size_t)(a.E + 1 + kWaves * a.E) * 4;
  balance_kernel<NV><<<dim3(a.blocks), dim3(kThreads), lds, s>>>(a);
  return hipGetLastError();
}

template <int NV>
hipError_t launch_grad_nv(const RouteGradArgs& a, hipStream_t s) {
  const uint32_t grid = std::min((a.T + 3) / 4, 2048u);
  route_grad_kernel<NV><<<dim3(grid), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

uint64_t balance_workspace_bytes(uint32_t T, uint32_t E) {
  const uint32_t blocks = balance_blocks(T);
  return blocks > 1 ? (uint64_t)blocks * 2 * (E + 1) * 4 : 0;
}

hipError_t launch_balance(const void* logits, bool bf16, const int32_t* ids, int32_t* counts, float* prob, float* loss,
                          void* workspace, float coef, uint32_t T, uint32_t E, uint32_t top_k, hipStream_t s) {
  const BalanceArgs a{logits, ids, counts, prob, loss, static_cast<uint32_t*>(workspace), coef, T, E, top_k,
                      balance_blocks(T), bf16};
  hipError_t e;
  if (E <= 64) e = launch_balance_nv<1>(a, s);
  else if (E <= 128) e = launch_balance_nv<2>(a, s);
  else if (E <= 192) e = launch_balance_nv<3>(a, s);
  else if (E <= 256) e = launch_balance_nv<4>(a, s);
  else e = launch_balance_nv<8>(a, s);
  if (e != hipSuccess || a.blocks == 1) return e;
  const uint32_t EB = E + 1, slices = kThreads / EB;  // E <= 512
  balance_sum_kernel<<<dim3(1), dim3(kThreads), (size_t)(1 + 2 * slices) * EB * 4, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_route_grad(const void* logits, bool bf16, const int32_t* ids, const float* dweights,
                             const int32_t* counts, const float* dloss, void* dlogits, float coef, uint32_t T,
                             uint32_t E, uint32_t top_k, bool renorm, hipStream_t s) {
  const RouteGradArgs a{logits, ids, dweights, counts, dloss, dlogits, coef, T, E, top_k, bf16, renorm};
  if (E <= 64) return launch_grad_nv<1>(a, s);
  if (E <= 128) return launch_grad_nv<2>(a, s);
  if (E <= 192) return launch_grad_nv<3>(a, s);
  if (E <= 256) return launch_grad_nv<4>(a, s);
  return launch_grad_nv<8>(a, s);
}

}  // namespace fp8q
