// Expert routing on gfx950: the top-k choice of each token with its softmax
// weights, the grouping of the chosen slots by expert, and the weighted sum of
// the experts' outputs back to the tokens.
//
//   ids[t][j]   = the j-th largest logit's index (ties: the lowest index first)
//   weight      = exp(l_j - l_max) / sum of exp(l - l_max) over the chosen
//                 experts, or over all of them
//   slot s      = t * top_k + j; order lists the slots sorted by expert
//                 (stable), slots without an expert last; pos is its inverse
//   offsets[e]  = number of slots with an expert below e
//
// Grouping is a counting sort.  Every wave owns a contiguous run of slots and
// counts them in LDS in slot order, so a slot's rank in its wave is the count
// it finds; wave counts, then block counts (through the workspace), then the
// exclusive sum over the experts give its place.  No atomics: the result is
// the stable order whatever the schedule.
#include <algorithm>

#include "quant_common.h"

namespace fp8q {
namespace {

constexpr uint32_t kWaves = 16, kThreads = 64 * kWaves;
// One workgroup routes up to this many tokens (or groups this many slots)
// alone: one launch.
constexpr uint32_t kLoneTokens = 64, kLoneSlots = 2048;
// Beyond, workgroups of at least this many tokens (slots), at most
// kMaxBlocks of them: the second launch's workgroups each sum all their counts.
constexpr uint32_t kBlockTokens = 32, kBlockSlots = 512, kMaxBlocks = 256;

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

// Exclusive sum over cnt[wave][e] in wave order, leaving the total in
// total[e]; then, for a lone workgroup, total[] becomes the exclusive sum over
// e.  EB = groups + 1 buckets (the last one: slots without a group).  Called by
// the whole workgroup.
__device__ __forceinline__ void sum_waves(uint32_t* cnt, uint32_t* total, uint32_t EB) {
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < EB; e += kThreads) {
    uint32_t run = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) {
      const uint32_t c = cnt[w * EB + e];
      cnt[w * EB + e] = run;
      run += c;
    }
    total[e] = run;
  }
  __syncthreads();
}

// total[0 .. EB) -> its exclusive sum, EB <= kThreads
__device__ __forceinline__ void scan_groups(uint32_t* total, uint32_t* wave_tot, uint32_t EB) {
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t v = tid < EB ? total[tid] : 0;
  uint32_t s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(s, d);
    if (lane >= (uint32_t)d) s += o;
  }
  if (lane == 63) wave_tot[wave] = s;
  __syncthreads();
  uint32_t before = 0;
  for (uint32_t w = 0; w < wave; ++w) before += wave_tot[w];
  if (tid < EB) total[tid] = before + s - v;
  __syncthreads();
}

// A wave's slots are few enough to stay in LDS (group and rank) up to this
// many; beyond, ids and pos hold them.
constexpr uint32_t kLdsSlots = 128;

// This wave's slots [s0, s1) of a lone workgroup: place = the stored rank + its
// wave's and its group's first place.
__device__ __forceinline__ void place_slots(const int32_t* ids, int32_t* order, int32_t* pos,
                                            const uint32_t* cnt, const uint32_t* base, uint32_t s0,
                                            uint32_t s1, uint32_t groups) {
  for (uint32_t s = s0 + (threadIdx.x & 63); s < s1; s += 64) {
    const uint32_t id = (uint32_t)ids[s], e = min(id, groups);
    const uint32_t p = (uint32_t)pos[s] + cnt[e] + base[e];
    pos[s] = (int32_t)p;
    order[p] = (int32_t)s;
  }
}

struct RouteArgs {
  const void* logits;
  int32_t *ids, *order, *pos, *offsets;
  float* weights;
  uint32_t* hist;  // [blocks][groups + 1]; unused by a lone workgroup
  uint32_t T, E, k, per_wave;  // tokens a wave
  bool bf16, renorm, lone;
};

// Each wave routes its tokens one after the other: lane l holds the logits
// l, l + 64, ...; each of the k rounds takes the wave's maximum and, of the
// positions that hold it, the lowest.  NV: logits a lane.  A lone workgroup
// finishes the grouping; otherwise pos holds ranks within the block and hist
// its counts.  Latency bound: k dependent rounds of about 20
// instructions.  16 tokens, 128 experts, top 8: 6.0 us with the grouping; 4576 tokens,
// 160 experts, top 6 (143 workgroups, two tokens a wave): 10.4-11 us, 0.17 TB/s.
template <int NV>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
  extern __shared__ uint32_t lds[];
  const uint32_t EB = a.E + 1;
  uint32_t *cnt = lds, *total = lds + kWaves * EB, *wave_tot = total + EB, *slots = wave_tot + kWaves;
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t first = ((uint64_t)blockIdx.x * kWaves + wave) * a.per_wave;
  const uint32_t t0 = (uint32_t)min(first, (uint64_t)a.T);
  const uint32_t t1 = (uint32_t)min(first + a.per_wave, (uint64_t)a.T);
  float raw[NV];  // the next token's logits
  auto load = [&](uint32_t t) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t e = 64 * i + lane;
      const uint64_t at = (uint64_t)t * a.E + min(e, a.E - 1);
      const float l = a.bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[at] << 16)
                             : static_cast<const float*>(a.logits)[at];
      raw[i] = e < a.E ? l : -INFINITY;
    }
  };
  if (t0 < t1) load(t0);
  for (uint32_t i = threadIdx.x; i < kWaves * EB; i += kThreads) cnt[i] = 0;
  __syncthreads();
  uint32_t* mine = cnt + wave * EB;
  slots += wave * kLdsSlots;
  const bool in_lds = a.per_wave * a.k <= kLdsSlots;
  for (uint32_t t = t0; t < t1; ++t) {
    uint32_t key[NV];
    float l[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      l[i] = clean_logit(raw[i]);
      key[i] = logit_key(l[i]);
    }
    load(min(t + 1, t1 - 1));
    uint32_t my_key = kNoKey, my_id = 0xFFFFFFFFu, top = kNoKey;  // lane j: the j-th choice
    for (uint32_t j = 0; j < a.k; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) best = max(best, key[i]);
      best = wave_max_u32(best);
      if (best == kNoKey) break;  // uniform: nothing left to choose
      uint32_t at = 0xFFFFFFFFu;
#pragma unroll
      for (int i = NV - 1; i >= 0; --i) {
        const uint64_t m = __builtin_amdgcn_ballot_w64(key[i] == best);
        if (m) at = 64 * i + (uint32_t)__builtin_ctzll(m);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (at == 64 * i + lane) key[i] = kNoKey;
      if (j == 0) top = best;
      if (lane == j) {
        my_key = best;
        my_id = at;
      }
    }
    const float lmax = top == kNoKey ? 0.0f : key_logit(top);
    const float ex = my_key == kNoKey ? 0.0f : exp_neg(key_logit(my_key) - lmax);
    float sum = ex;
    if (!a.renorm) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) sum += l[i] == -INFINITY ? 0.0f : exp_neg(l[i] - lmax);
    }
    sum = wave_sum_f32(sum);
    // ranks within the wave: a token's experts differ, so every counter has
    // one lane; its slots without an expert follow one another
    const bool on = lane < a.k, none = on && my_id == 0xFFFFFFFFu;
    const uint64_t nones = __builtin_amdgcn_ballot_w64(none);
    if (on) {
      const uint64_t s = (uint64_t)t * a.k + lane;
      a.ids[s] = (int32_t)my_id;
      a.weights[s] = my_key == kNoKey ? 0.0f : ex / sum;
      const uint32_t e = none ? a.E : my_id, c = mine[e];
      const uint32_t rank = none ? c + (uint32_t)__builtin_popcountll(nones & ((1ull << lane) - 1)) : c;
      if (in_lds)
        slots[(t - t0) * a.k + lane] = rank << 16 | e;  // rank < kLdsSlots
      else
        a.pos[s] = (int32_t)rank;
      if (!none) mine[e] = c + 1;
    }
    if (lane == 0 && nones) mine[a.E] += (uint32_t)__builtin_popcountll(nones);
    __builtin_amdgcn_wave_barrier();
  }
  sum_waves(cnt, total, EB);
  if (a.lone) {
    scan_groups(total, wave_tot, EB);
    for (uint32_t e = threadIdx.x; e < EB; e += kThreads) a.offsets[e] = (int32_t)total[e];
  } else {
    for (uint32_t e = threadIdx.x; e < EB; e += kThreads) a.hist[blockIdx.x * EB + e] = total[e];
  }
  // places (a lone workgroup) or ranks within the block
  for (uint32_t i = lane; i < (t1 - t0) * a.k; i += 64) {
    const uint32_t s = t0 * a.k + i;
    uint32_t rank, e;
    if (in_lds) {
      rank = slots[i] >> 16;
      e = slots[i] & 0xFFFF;
    } else {
      rank = (uint32_t)a.pos[s];
      e = min((uint32_t)a.ids[s], a.E);
    }
    rank += mine[e] + (a.lone ? total[e] : 0);
    a.pos[s] = (int32_t)rank;
    if (a.lone) a.order[rank] = (int32_t)s;
  }
}

// The first half for given ids: each wave counts its slots 64 at a time; the
// lanes that hold the same group find one another bit by bit.  Latency of its few
// steps a wave: 2048 slots of 64 groups alone 4.9 us; with the placing launch, 27456 of
// 160: 3.6 + 5.6 us, 2^20 of 64: 7.5 + 11.1, 2^20 of 512: 8.8 + 26.1 (there each workgroup's
// sum over the 256 x 513 counts; 24 MB of ids, ranks and places take 5).
__global__ __launch_bounds__(kThreads) void count_kernel(const int32_t* ids, int32_t* order,
                                                         int32_t* pos, int32_t* offsets,
                                                         uint32_t* hist, uint32_t n, uint32_t groups,
                                                         uint32_t bits, uint32_t per_wave, bool lone) {
  extern __shared__ uint32_t lds[];
  const uint32_t EB = groups + 1;
  uint32_t *cnt = lds, *total = lds + kWaves * EB, *wave_tot = total + EB;
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (uint32_t i = threadIdx.x; i < kWaves * EB; i += kThreads) cnt[i] = 0;
  __syncthreads();
  uint32_t* mine = cnt + wave * EB;
  const uint64_t first = ((uint64_t)blockIdx.x * kWaves + wave) * per_wave;
  const uint32_t s0 = (uint32_t)min(first, (uint64_t)n), s1 = (uint32_t)min(first + per_wave, (uint64_t)n);
  for (uint32_t b = s0; b < s1; b += 64) {
    const uint32_t s = b + lane;
    const bool on = s < s1;
    const uint32_t e = on ? min((uint32_t)ids[s], groups) : 0;
    uint64_t same = __builtin_amdgcn_ballot_w64(on);
    for (uint32_t i = 0; i < bits; ++i) {
      const uint64_t m = __builtin_amdgcn_ballot_w64((e >> i) & 1);
      same &= ((e >> i) & 1) ? m : ~m;
    }
    if (on) {
      const uint32_t c = mine[e];
      pos[s] = (int32_t)(c + (uint32_t)__builtin_popcountll(same & ((1ull << lane) - 1)));
      __builtin_amdgcn_wave_barrier();
      if ((same >> lane) == 1) mine[e] = c + (uint32_t)__builtin_popcountll(same);  // its last lane
    }
    __builtin_amdgcn_wave_barrier();
  }
  sum_waves(cnt, total, EB);
  if (lone) {
    scan_groups(total, wave_tot, EB);
    for (uint32_t e = threadIdx.x; e < EB; e += kThreads) offsets[e] = (int32_t)total[e];
    place_slots(ids, order, pos, mine, total, s0, s1, groups);
  } else {
    for (uint32_t s = s0 + lane; s < s1; s += 64) pos[s] += (int32_t)mine[min((uint32_t)ids[s], groups)];
    for (uint32_t e = threadIdx.x; e < EB; e += kThreads) hist[blockIdx.x * EB + e] = total[e];
  }
}

// The second half of a grouping by many workgroups: workgroup b adds, for
// every group, the counts of the blocks before b and those of all groups before,
// and places its slots.  The threads are dealt as EB columns x parts of the
// blocks' rows.  27456 slots of 160 experts: 5.9 us, latency of the count sums.
__global__ __launch_bounds__(kThreads) void place_kernel(const int32_t* ids, int32_t* order,
                                                         int32_t* pos, int32_t* offsets,
                                                         const uint32_t* hist, uint32_t n,
                                                         uint32_t groups, uint32_t per_block) {
  extern __shared__ uint32_t lds[];
  const uint32_t EB = groups + 1, nb = gridDim.x, b = blockIdx.x;
  uint32_t *total = lds, *before = lds + EB, *wave_tot = before + EB, *zero = wave_tot + kWaves;
  constexpr uint32_t kAhead = 16;
  const uint32_t parts = kThreads / EB;  // >= 1: groups < kThreads
  const uint32_t e = threadIdx.x % EB, part = threadIdx.x / EB;
  uint32_t *pt = zero + EB, *pb = pt + kThreads;  // partial sums per thread
  if (part < parts) {
    uint32_t st = 0, sb = 0;
    // all of a thread's counts in flight at once (kMaxBlocks of them at most)
    for (uint32_t r0 = part; r0 < nb; r0 += kAhead * parts) {
      uint32_t c[kAhead];
#pragma unroll
      for (uint32_t i = 0; i < kAhead; ++i) c[i] = hist[min(r0 + i * parts, nb - 1) * EB + e];
#pragma unroll
      for (uint32_t i = 0; i < kAhead; ++i) {
        const uint32_t r = r0 + i * parts;
        st += r < nb ? c[i] : 0;
        sb += r < b ? c[i] : 0;
      }
    }
    pt[threadIdx.x] = st;
    pb[threadIdx.x] = sb;
  }
  __syncthreads();
  if (threadIdx.x < EB) {
    uint32_t st = 0, sb = 0;
    for (uint32_t q = 0; q < parts; ++q) {
      st += pt[q * EB + threadIdx.x];
      sb += pb[q * EB + threadIdx.x];
    }
    total[threadIdx.x] = st;
    before[threadIdx.x] = sb;
  }
  __syncthreads();
  scan_groups(total, wave_tot, EB);
  if (threadIdx.x < EB) {
    if (b == 0) offsets[threadIdx.x] = (int32_t)total[threadIdx.x];
    total[threadIdx.x] += before[threadIdx.x];
  }
  __syncthreads();
  const uint64_t first = (uint64_t)b * per_block;
  const uint32_t s0 = (uint32_t)min(first, (uint64_t)n), s1 = (uint32_t)min(first + per_block, (uint64_t)n);
  for (uint32_t s = s0 + threadIdx.x; s < s1; s += kThreads) {
    const uint32_t p = (uint32_t)pos[s] + total[min((uint32_t)ids[s], groups)];
    pos[s] = (int32_t)p;
    order[p] = (int32_t)s;
  }
}

// out[t] = bf16( sum over j, in order, of weights[t][j] * y[pos[t][j]] ); slots
// without an expert, or past the R rows of y whatever the plan holds, add
// nothing.  Eight columns per thread, summed in fp32.  Bound
// by reading y: T = 4576, top 4, H = 5120: 38 us, 6.2 TB/s read and written.
__global__ __launch_bounds__(256) void combine_kernel(const uint16_t* __restrict__ y,
                                                      const float* __restrict__ weights,
                                                      const int32_t* __restrict__ pos,
                                                      const int32_t* __restrict__ offsets,
                                                      uint16_t* __restrict__ out, uint32_t R, uint32_t E,
                                                      uint32_t k, uint32_t H, uint32_t blocks_h) {
  const uint32_t t = blockIdx.y * (gridDim.x / blocks_h) + blockIdx.x / blocks_h;
  const uint32_t h = (blockIdx.x % blocks_h) * 2048 + threadIdx.x * 8;
  if (t >= R / k || h >= H) return;
  const uint32_t taken = min((uint32_t)offsets[E], R);
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (uint32_t j = 0; j < k; ++j) {
    const uint32_t p = (uint32_t)pos[(uint64_t)t * k + j];
    if (p >= taken) continue;
    const float w = weights[(uint64_t)t * k + j];
    const u32x4 v = *reinterpret_cast<const u32x4*>(y + (uint64_t)p * H + h);
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[2 * i] = __builtin_fmaf(w, bf_lo(d[i]), s[2 * i]);
      s[2 * i + 1] = __builtin_fmaf(w, bf_hi(d[i]), s[2 * i + 1]);
    }
  }
  u32x4 o;
  o.x = bf16_bits_rne(s[0]) | (bf16_bits_rne(s[1]) << 16);
  o.y = bf16_bits_rne(s[2]) | (bf16_bits_rne(s[3]) << 16);
  o.z = bf16_bits_rne(s[4]) | (bf16_bits_rne(s[5]) << 16);
  o.w = bf16_bits_rne(s[6]) | (bf16_bits_rne(s[7]) << 16);
  *reinterpret_cast<u32x4*>(out + (uint64_t)t * H + h) = o;
}

uint32_t count_lds(uint32_t groups) { return (kWaves * (groups + 1) + (groups + 1) + kWaves) * 4; }
uint32_t route_lds(uint32_t groups) { return count_lds(groups) + kWaves * kLdsSlots * 4; }
uint32_t place_lds(uint32_t groups) { return (3 * (groups + 1) + kWaves + 2 * kThreads) * 4; }

// tokens (slots) a wave and workgroups for n of them
void split_work(uint64_t n, uint32_t lone, uint32_t block, uint32_t& per_wave, uint32_t& blocks) {
  if (n <= lone) {
    per_wave = (uint32_t)((n + kWaves - 1) / kWaves);
    blocks = 1;
  } else {
    const uint64_t per_block = std::max<uint64_t>(block, (n + kMaxBlocks - 1) / kMaxBlocks);
    per_wave = (uint32_t)((per_block + kWaves - 1) / kWaves);
    blocks = (uint32_t)((n + (uint64_t)per_wave * kWaves - 1) / ((uint64_t)per_wave * kWaves));
  }
}

hipError_t launch_place(const int32_t* ids, int32_t* order, int32_t* pos, int32_t* offsets,
                        const uint32_t* hist, uint32_t n, uint32_t groups, uint32_t per_block,
                        uint32_t blocks, hipStream_t s) {
  place_kernel<<<dim3(blocks), dim3(kThreads), place_lds(groups), s>>>(ids, order, pos, offsets, hist,
                                                                       n, groups, per_block);
  return hipGetLastError();
}

}  // namespace

uint64_t route_workspace_bytes(uint32_t T, uint32_t E) {
  uint32_t per_wave, blocks;
  split_work(T, kLoneTokens, kBlockTokens, per_wave, blocks);
  return blocks > 1 ? (uint64_t)blocks * (E + 1) * 4 : 0;
}

uint64_t group_workspace_bytes(uint32_t n, uint32_t groups) {
  uint32_t per_wave, blocks;
  split_work(n, kLoneSlots, kBlockSlots, per_wave, blocks);
  return blocks > 1 ? (uint64_t)blocks * (groups + 1) * 4 : 0;
}

hipError_t launch_route(const void* logits, bool bf16, int32_t* ids, float* weights, int32_t* order,
                        int32_t* pos, int32_t* offsets, void* workspace, uint32_t T, uint32_t E,
                        uint32_t top_k, bool renorm, hipStream_t s) {
  uint32_t per_wave, blocks;
  split_work(T, kLoneTokens, kBlockTokens, per_wave, blocks);
  RouteArgs a{logits, ids, order, pos, offsets, weights, static_cast<uint32_t*>(workspace), T, E,
              top_k, per_wave, bf16, renorm, blocks == 1};
  const dim3 grid(blocks), block(kThreads);
  const uint32_t lds = route_lds(E);
  if (E <= 64) route_kernel<1><<<grid, block, lds, s>>>(a);
  else if (E <= 128) route_kernel<2><<<grid, block, lds, s>>>(a);
  else if (E <= 256) route_kernel<4><<<grid, block, lds, s>>>(a);
  else route_kernel<8><<<grid, block, lds, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || blocks == 1) return e;
  return launch_place(ids, order, pos, offsets, a.hist, T * top_k, E, per_wave * kWaves * top_k, blocks, s);
}

hipError_t launch_group_rows(const int32_t* ids, int32_t* order, int32_t* pos, int32_t* offsets,
                             void* workspace, uint32_t n, uint32_t groups, hipStream_t s) {
  uint32_t per_wave, blocks, bits = 0;
  split_work(n, kLoneSlots, kBlockSlots, per_wave, blocks);
  per_wave = (per_wave + 63) / 64 * 64;  // whole waves of slots; later blocks may then be empty
  while ((groups >> bits) != 0) ++bits;
  count_kernel<<<dim3(blocks), dim3(kThreads), count_lds(groups), s>>>(
      ids, order, pos, offsets, static_cast<uint32_t*>(workspace), n, groups, bits, per_wave, blocks == 1);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || blocks == 1) return e;
  return launch_place(ids, order, pos, offsets, static_cast<uint32_t*>(workspace), n, groups,
                      per_wave * kWaves, blocks, s);
}

hipError_t launch_combine(const uint16_t* y, const float* weights, const int32_t* pos,
                          const int32_t* offsets, uint16_t* out, uint32_t T, uint32_t E,
                          uint32_t top_k, uint32_t H, hipStream_t s) {
  // a launch holds fewer than 2^32 threads a dimension: 2^23 workgroups here, the
  // tokens beyond in y (T * blocks_h < 2^30)
  const uint32_t blocks_h = (uint32_t)(((uint64_t)H + 2047) / 2048);
  const uint32_t tokens = std::min(T, (1u << 23) / blocks_h);
  combine_kernel<<<dim3(tokens * blocks_h, (T + tokens - 1) / tokens), dim3(256), 0, s>>>(
      y, weights, pos, offsets, out, T * top_k, E, top_k, H, blocks_h);
  return hipGetLastError();
}

}  // namespace fp8q
