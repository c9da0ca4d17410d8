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
// A wave takes four tokens at a time, one a 16-lane row, lane l of it holding the logits
// l, l + 16, ...: a reduction is four DPP steps for all four.  (One token a wave, its
// reductions over 64 lanes: 13 us a launch at 16384 tokens of 160 experts, twice the
// present.)  Probabilities are summed in registers, then
// over a workgroup's waves and over the workgroups in a fixed order; counts are integers,
// so their LDS atomics give the same result in any order.  16384 tokens of 160 experts, bf16
// (5 MB, in the caches): 7.7 us, the sums' kernel 5.8, the gradient's 9.4, of which a launch
// is 2.3 each; 25 tokens of 64: 3.1 and 3.6, one launch each.  Bound by the latency of the
// loads: at 16384 tokens a wave makes one pass of its loop, and of its cycles 71% wait in the
// loss's kernel and 64% in the gradient's, where 18% and 22% issue.
#include <algorithm>

#include "wave_common.h"

namespace fp8q {
namespace {

constexpr uint32_t kWaves = 16, kThreads = 64 * kWaves;
// One workgroup takes up to this many tokens alone (one launch; 128 tokens of 160 experts: 7.5
// us, 8.6 by two, but 256: 11.2 and 8.8); beyond, at least kBlockTokens a workgroup and at
// most kMaxBlocks of them (128 or 512 at 16384 tokens: within 2%), summed by a second launch.
constexpr uint32_t kLoneTokens = 128, kBlockTokens = 64, kMaxBlocks = 256;
// Slices of that sum, each joined behind the one before: of 256 workgroups 16 leave a thread
// one round of 16 loads.  (As many as the threads make, 204 at 8 experts: 9.2 us a call and not
// 6.5 at 16384 tokens; 93 at 40: 8.0 and not 7.3.)
constexpr uint32_t kMaxSlices = 16;

uint32_t balance_blocks(uint32_t T) {
  return T <= kLoneTokens ? 1 : std::min((T + kBlockTokens - 1) / kBlockTokens, kMaxBlocks);
}

__device__ __forceinline__ float dpp_row_sum_f32(float v) {
  v += dpp_f32<0xB1>(v);
  v += dpp_f32<0x4E>(v);
  v += dpp_f32<0x141>(v);
  return v + dpp_f32<0x140>(v);
}

// This lane's logits of token t (the row's) as fp32; -inf where there is none or NaN.
template <int NV>
__device__ __forceinline__ void load_logits(const void* logits, bool bf16, uint32_t t, uint32_t E, uint32_t l16,
                                            float (&l)[NV]) {
  const uint64_t at = (uint64_t)t * E + l16;
  if (bf16) {  // uniform
    const uint16_t* p = static_cast<const uint16_t*>(logits) + at;
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = 16 * i + l16 < E ? __uint_as_float((uint32_t)p[16 * i] << 16) : -INFINITY;
  } else {
    const float* p = static_cast<const float*>(logits) + at;
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = 16 * i + l16 < E ? p[16 * i] : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) l[i] = clean_logit(l[i]);
}

// The key of the row's largest logit.
template <int NV>
__device__ __forceinline__ uint32_t top_key(const float (&l)[NV]) {
  float top = l[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) top = fmaxf(top, l[i]);
  return dpp_row_max_u32(logit_key(top));
}

// e[i] = e^(l[i] - top), 0 where l is -inf; returns the row's sum (0: nothing to choose).
template <int NV>
__device__ __forceinline__ float exp_logits(const float (&l)[NV], uint32_t top, float (&e)[NV]) {
  const float lmax = top == kNoKey ? 0.0f : key_logit(top);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    e[i] = l[i] == -INFINITY ? 0.0f : exp_neg(l[i] - lmax);
    sum += e[i];
  }
  return dpp_row_sum_f32(sum);
}

// A workgroup's sums, whole 16-byte words.
__host__ __device__ constexpr uint32_t part_words(uint32_t E) { return (2 * (E + 1) + 3) / 4 * 4; }

struct BalanceArgs {
  const void* logits;
  const int32_t* ids;
  int32_t* counts;  // [E + 1], the last one n
  float *prob, *loss;
  uint32_t* part;  // [blocks][part_words(E)]: E + 1 probability sums, E + 1 counts; not a lone workgroup's
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
  const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, row = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (uint32_t e = threadIdx.x; e <= a.E; e += kThreads) cnt[e] = 0;
  __syncthreads();
  float acc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.0f;
  uint32_t n = 0;  // of the row's tokens, those with an expert
  for (uint64_t t0 = (uint64_t)(blockIdx.x * kWaves + wave) * 4; t0 < a.T; t0 += (uint64_t)gridDim.x * kWaves * 4) {
    const bool live = t0 + row < a.T;  // (rows past the last token repeat it and count nothing)
    const uint32_t t = (uint32_t)min(t0 + row, (uint64_t)a.T - 1);
    float l[NV], x[NV];
    load_logits<NV>(a.logits, a.bf16, t, a.E, l16, l);
    uint32_t id[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      id[j] = live && 16 * j + l16 < a.k ? (uint32_t)a.ids[(uint64_t)t * a.k + 16 * j + l16] : a.E;
    const float sum = exp_logits<NV>(l, top_key<NV>(l), x);
    const float r = live && sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = __builtin_fmaf(x[i], r, acc[i]);
    n += live && sum > 0.0f ? 1 : 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (id[j] < a.E) atomicAdd(&cnt[id[j]], 1u);
  }
  if (l16 == 0 && n) atomicAdd(&cnt[a.E], n);
#pragma unroll
  for (int i = 0; i < NV; ++i) {  // the four rows
    acc[i] += __shfl_xor(acc[i], 16);
    acc[i] += __shfl_xor(acc[i], 32);
    if (row == 0 && 16 * i + l16 < a.E) sums[wave * a.E + 16 * i + l16] = acc[i];
  }
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
    uint32_t* out = a.part + (uint64_t)blockIdx.x * part_words(a.E);
    for (uint32_t e = threadIdx.x; e <= a.E; e += kThreads) {
      out[e] = e < a.E ? __float_as_uint(sums[e]) : 0;
      out[a.E + 1 + e] = cnt[e];
    }
  }
}

// The workgroups' sums: `slices` slices of the workgroups, each in order, then in slice
// order.  One workgroup, bound by the latency of its loads: up to 16 of 16 bytes in flight a
// thread.  (Words past the counts are never used.)  Both launches of a call, bf16 logits, us,
// with 24 in flight -> 16: 1024 tokens of 8 experts 6.3 -> 5.8, 64: 7.1 -> 6.8, 160: 9.3 -> 8.7,
// 256: 11.1 -> 10.5; 16384 tokens of 64: 7.9 -> 7.7, 128: 10.5 -> 10.8, 160: 11.5 -> 11.7, 192:
// 13.5 -> 12.6, 256: 16.0 both.
__global__ __launch_bounds__(kThreads) void balance_sum_kernel(BalanceArgs a, uint32_t slices) {
  extern __shared__ uint32_t lds[];  // [slices][part_words(E)], then psum and cnt in slice 0's place
  __shared__ float red[kWaves];
  constexpr uint32_t kInFlight = 16;
  const uint32_t EB = a.E + 1, R = part_words(a.E), V = R / 4;
  const u32x4* part = reinterpret_cast<const u32x4*>(a.part);
  for (uint32_t at = threadIdx.x; at < slices * V; at += kThreads) {
    const uint32_t slice = at / V, c = at % V;
    float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 n = {0, 0, 0, 0};
    for (uint32_t b0 = slice; b0 < a.blocks; b0 += kInFlight * slices) {
      u32x4 v[kInFlight];
#pragma unroll
      for (uint32_t i = 0; i < kInFlight; ++i)
        v[i] = b0 + i * slices < a.blocks ? part[(uint64_t)(b0 + i * slices) * V + c] : u32x4{0, 0, 0, 0};
#pragma unroll
      for (uint32_t i = 0; i < kInFlight; ++i) {
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) p[j] += __uint_as_float(v[i][j]);
        n += v[i];
      }
    }
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) lds[slice * R + 4 * c + j] = 4 * c + j < EB ? __float_as_uint(p[j]) : n[j];
  }
  __syncthreads();
  for (uint32_t c = threadIdx.x; c < R; c += kThreads) {
    float p = 0.0f;
    uint32_t n = 0;
    for (uint32_t s = 0; s < slices; ++s) {
      p += __uint_as_float(lds[s * R + c]);
      n += lds[s * R + c];
    }
    lds[c] = c < EB ? __float_as_uint(p) : n;
  }
  __syncthreads();
  finish(a, reinterpret_cast<const float*>(lds), lds + EB, red);
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

constexpr uint32_t kGradWaves = 4, kGradGrid = 1024;

// Keeps the compiler from moving LDS accesses across.
__device__ __forceinline__ void lds_order() {
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

template <int NV>
__global__ __launch_bounds__(64 * kGradWaves) void route_grad_kernel(RouteGradArgs a) {
  extern __shared__ uint32_t lds[];  // a row: [E] sums of dweights, [E] slots
  const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, row = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* dsum = reinterpret_cast<float*>(lds) + (size_t)(wave * 4 + row) * 2 * a.E;
  uint32_t* slots = reinterpret_cast<uint32_t*>(dsum) + a.E;
  float share[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) share[i] = 0.0f;
  if (a.counts) {
    const float n = (float)a.counts[a.E];
    const float f = n > 0.0f ? a.coef * (float)a.E / (n * (float)a.k) / n * (a.dloss ? *a.dloss : 1.0f) : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float c = (float)a.counts[min(16 * i + l16, a.E - 1)];
      share[i] = n > 0.0f && 16 * i + l16 < a.E ? f * c : 0.0f;
    }
  }
  for (uint64_t t0 = (uint64_t)(blockIdx.x * kGradWaves + wave) * 4; t0 < a.T;
       t0 += (uint64_t)gridDim.x * kGradWaves * 4) {
    const bool live = t0 + row < a.T;  // (rows past the last token repeat it and store nothing)
    const uint32_t t = (uint32_t)min(t0 + row, (uint64_t)a.T - 1);
    float l[NV], x[NV], g[NV];
    load_logits<NV>(a.logits, a.bf16, t, a.E, l16, l);
    uint32_t id[2];
    float dwj[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool slot = a.ids && 16 * j + l16 < a.k;
      id[j] = slot ? (uint32_t)a.ids[(uint64_t)t * a.k + 16 * j + l16] : a.E;
      dwj[j] = id[j] < a.E ? a.dweights[(uint64_t)t * a.k + 16 * j + l16] : 0.0f;
    }
    const uint32_t top = top_key<NV>(l);
    const float sum = exp_logits<NV>(l, top, x);
    const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) dot = __builtin_fmaf(x[i] * r, share[i], dot);
    dot = dpp_row_sum_f32(dot);
#pragma unroll
    for (int i = 0; i < NV; ++i) g[i] = x[i] * r * (share[i] - dot);
    if (a.ids) {
      // the slots' gradients and number at their experts, through the row's part of LDS (a
      // wave's LDS accesses are in order)
      float d[NV], m[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (16 * i + l16 < a.E) {
          dsum[16 * i + l16] = 0.0f;
          if (a.renorm) slots[16 * i + l16] = 0;
        }
      lds_order();
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (id[j] < a.E) {
          unsafeAtomicAdd(&dsum[id[j]], dwj[j]);
          if (a.renorm) atomicAdd(&slots[id[j]], 1u);
        }
      lds_order();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = 16 * i + l16 < a.E;
        d[i] = in ? dsum[min(16 * i + l16, a.E - 1)] : 0.0f;
        m[i] = !a.renorm ? 1.0f : in ? (float)slots[min(16 * i + l16, a.E - 1)] : 0.0f;
      }
      lds_order();
      float rw = r;
      if (a.renorm) {
        // over the chosen slots alone, with their own maximum: chosen by another
        // rule than the largest logits, they may all lie far below the top
        float c[NV], mass = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] = m[i] > 0.0f ? l[i] : -INFINITY;
        const uint32_t top_c = top_key<NV>(c);
        if (__builtin_amdgcn_ballot_w64(top_c != top)) exp_logits<NV>(c, top_c, x);  // (equal tops: equal values)
#pragma unroll
        for (int i = 0; i < NV; ++i) mass = __builtin_fmaf(x[i], m[i], mass);
        mass = dpp_row_sum_f32(mass);
        rw = mass > 0.0f ? 1.0f / mass : 0.0f;
      }
      float wd = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) wd = __builtin_fmaf(x[i] * rw, d[i], wd);
      wd = dpp_row_sum_f32(wd);
#pragma unroll
      for (int i = 0; i < NV; ++i) g[i] += x[i] * rw * (d[i] - m[i] * wd);
    }
    // an expert that cannot be chosen: 0, and not 0 * (a NaN or infinite gradient)
#pragma unroll
    for (int i = 0; i < NV; ++i) g[i] = l[i] == -INFINITY ? 0.0f : g[i];
    if (live) {
      const uint64_t at = (uint64_t)t * a.E + l16;
      if (a.bf16) {
        uint16_t* p = static_cast<uint16_t*>(a.dlogits) + at;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (16 * i + l16 < a.E) p[16 * i] = bf16_rne(g[i]);
      } else {
        float* p = static_cast<float*>(a.dlogits) + at;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (16 * i + l16 < a.E) p[16 * i] = g[i];
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
  const uint32_t grid = std::min((a.T + 4 * kGradWaves - 1) / (4 * kGradWaves), kGradGrid);
  const size_t lds = a.ids ? (size_t)kGradWaves * 4 * 2 * a.E * 4 : 0;  // 64 KB at 512 experts
  route_grad_kernel<NV><<<dim3(grid), dim3(64 * kGradWaves), lds, s>>>(a);
  return hipGetLastError();
}

// f(NV) for the logits a lane holds: 2 for each 32 experts up to 256, then 8 for each 128.  (In
// the next larger instance, the gradient of 16384 tokens, bf16: 96 experts 5.4 us and not 5.0,
// 224: 12.2 and not 8.5, 384: 22.9 and not 19.7.)
template <class F>
hipError_t for_experts(uint32_t E, F&& f) {
  using std::integral_constant;
  if (E > 384) return f(integral_constant<int, 32>{});
  if (E > 256) return f(integral_constant<int, 24>{});
  switch ((E + 31) / 32) {
    case 1: return f(integral_constant<int, 2>{});
    case 2: return f(integral_constant<int, 4>{});
    case 3: return f(integral_constant<int, 6>{});
    case 4: return f(integral_constant<int, 8>{});
    case 5: return f(integral_constant<int, 10>{});
    case 6: return f(integral_constant<int, 12>{});
    case 7: return f(integral_constant<int, 14>{});
    default: return f(integral_constant<int, 16>{});
  }
}

}  // namespace

uint64_t balance_workspace_bytes(uint32_t T, uint32_t E) {
  const uint32_t blocks = balance_blocks(T);
  return blocks > 1 ? (uint64_t)blocks * part_words(E) * 4 : 0;
}

hipError_t launch_balance(const void* logits, bool bf16, const int32_t* ids, int32_t* counts, float* prob, float* loss,
                          void* workspace, float coef, uint32_t T, uint32_t E, uint32_t top_k, hipStream_t s) {
  const BalanceArgs a{logits, ids, counts, prob, loss, static_cast<uint32_t*>(workspace), coef, T, E, top_k,
                      balance_blocks(T), bf16};
  const hipError_t e = for_experts(E, [&](auto nv) { return launch_balance_nv<decltype(nv)::value>(a, s); });
  if (e != hipSuccess || a.blocks == 1) return e;
  const uint32_t R = part_words(E), slices = std::clamp(kThreads / (R / 4), 1u, kMaxSlices);
  balance_sum_kernel<<<dim3(1), dim3(kThreads), (size_t)slices * R * 4, s>>>(a, slices);
  return hipGetLastError();
}

hipError_t launch_route_grad(const void* logits, bool bf16, const int32_t* ids, const float* dweights,
                             const int32_t* counts, const float* dloss, void* dlogits, float coef, uint32_t T,
                             uint32_t E, uint32_t top_k, bool renorm, hipStream_t s) {
  const RouteGradArgs a{logits, ids, dweights, counts, dloss, dlogits, coef, T, E, top_k, bf16, renorm};
  return for_experts(E, [&](auto nv) { return launch_grad_nv<decltype(nv)::value>(a, s); });
}

}  // namespace fp8q
