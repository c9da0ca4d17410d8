// Low-rank adapters beside a shared projection: the epilogue that adds a row's
// adapter to the GEMM's fp32 accumulators (lora.hip holds the kernels).
#pragma once

#include "mfma_common.h"

namespace fp8q {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// v = x . A^T in kLoraParts contiguous parts of K at most, [M][parts][ld] fp32
// (ld: the rank rounded up to 32, zero beyond it).
constexpr uint32_t kLoraMaxParts = 4;

struct LoraArgs {
  const float* v;         // [M][parts][ld]
  const uint16_t* b;      // [adapters][N][rank] bf16
  const float* scale;     // [adapters]
  const int32_t* ids;     // [M]; outside 0 .. adapters-1: no adapter
  uint32_t adapters, rank, ld, parts, N;
};

__device__ __forceinline__ uint32_t lora_id(const LoraArgs& a, uint32_t m) {
  const uint32_t id = (uint32_t)a.ids[m];
  return id < a.adapters ? id : 0xFFFFFFFFu;
}

__device__ __forceinline__ v4f mfma_bf16_32(const u32x4& w, const u32x4& x, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, x), c, 0,
                                                 0, 0);
}

// v * s as the sum of two bf16 numbers (its rounding and the rest), four at a time
__device__ __forceinline__ void split_bf16(const v4f& v, float s, uint2& hi, uint2& lo) {
  uint32_t h[4], r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = v[i] * s;
    h[i] = bf16_rne(f);
    r[i] = bf16_rne(f - __uint_as_float(h[i] << 16));
  }
  hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  lo = make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// out[m, n] += scale[a] * sum_r v[m, r] * B[a][n, r] for the rows m of adapter
// a, on the GEMM's accumulator layout (lane l: row l % 16 of its 16-row tile,
// columns 4 * (l / 16) .. +3).  A wave walks the distinct adapters of its rows
// (up to 64, a row a lane); for each, one pass over the rank in MFMA steps of 32,
// whose result only that adapter's rows take: the others keep their accumulators
// (a zero v would not do: an adapter's infinities would reach them).  The scaled
// v enters the bf16 product as the sum of two bf16 numbers, so that the delta
// keeps about 16 bits of v, and the accumulator is rounded once, with the base.
// Bound by reading B at decode (25 rows of 22 adapters, N = 17408, rank 64: 49 MB in
// 13 us beside the base's 26); at prompts 15-25 us of the GEMM's 400 (M = 4576, N
// = 5120, K = 17408, rank 32).
struct LoraEpilogue {
  LoraArgs a;

  // The items (adapter, rank step of 32) of up to 64 rows, dealt over `stride`
  // participants of which this is `first`.
  struct Items {
    uint32_t id, steps, first, stride;  // id: of row m0 + lane
    uint64_t left, mine = 0;            // rows not yet visited; rows of the current adapter
    uint32_t turn = 0, step = 0, ad = 0;
    __device__ __forceinline__ bool next() {
      while (true) {
        if (mine == 0) {
          if (left == 0) return false;
          ad = (uint32_t)__builtin_amdgcn_readlane((int)id, __builtin_ctzll(left));
          mine = __builtin_amdgcn_ballot_w64(id == ad);
          left &= ~mine;
          step = 0;
        } else if (++step == steps) {
          mine = 0;
          continue;
        }
        if (turn++ % stride == first) return true;
      }
    }
  };
  template <int TM>
  __device__ __forceinline__ Items items(uint32_t m0, uint32_t M, uint32_t lane, uint32_t first,
                                         uint32_t stride) const {
    static_assert(TM <= 4, "a row a lane");
    Items it;
    it.id = lane < 16 * TM && m0 + lane < M ? lora_id(a, m0 + lane) : 0xFFFFFFFFu;
    it.left = __builtin_amdgcn_ballot_w64(it.id != 0xFFFFFFFFu);
    it.steps = (a.rank + 31) / 32;
    it.first = __builtin_amdgcn_readfirstlane(first);  // (uniform over the wave: keeps the walk scalar)
    it.stride = stride;
    return it;
  }

  // B fragments of one item: TN column tiles from n0 on, this lane's 8 ranks at k
  template <int TN>
  __device__ __forceinline__ void load_b(u32x4 (&b)[TN], uint32_t ad, uint32_t k, uint32_t n0,
                                         uint32_t l16) const {
    const uint16_t* from = a.b + (uint64_t)ad * a.N * a.rank + min(k, a.rank - 8);
#pragma unroll
    for (int t = 0; t < TN; ++t)  // past the columns: any in-bounds values, not used
      b[t] = *reinterpret_cast<const u32x4*>(from + (uint64_t)min(n0 + 16 * t + l16, a.N - 1) * a.rank);
  }
  template <int TN>
  __device__ __forceinline__ void zero_past_rank(u32x4 (&b)[TN], uint32_t k) const {
    if (k >= a.rank) {
#pragma unroll
      for (int t = 0; t < TN; ++t) b[t] = u32x4{0, 0, 0, 0};
    }
  }

  // acc += b . (hi + lo) for the lanes of rows that are `own`
  template <int TN, class Acc>
  __device__ __forceinline__ void accumulate(Acc&& acc, int tm, const u32x4 (&b)[TN], const u32x4& hi,
                                             const u32x4& lo, bool own) const {
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      const v4f sum = mfma_bf16_32(b[t], hi, mfma_bf16_32(b[t], lo, acc(tm, t)));
#pragma unroll
      for (int i = 0; i < 4; ++i) acc(tm, t)[i] = own ? sum[i] : acc(tm, t)[i];
    }
  }

  // Many rows (prompts: one or two adapters a wave): the wave takes its own
  // rows' adapters one after another, v read where it is used.
  template <int TM, int TN, class Acc>
  __device__ __forceinline__ void add(Acc&& acc, uint32_t m0, uint32_t n0, uint32_t M, uint32_t lane,
                                      uint32_t split) const {
    if (split != 0) return;  // split-K: the first part adds
    const uint32_t l16 = lane & 15, q = lane >> 4;
    Items it = items<TM>(m0, M, lane, 0, 1);
    while (it.next()) {
      const uint32_t k = 32 * it.step + 8 * q;
      const float s = a.scale[it.ad];
      u32x4 b[TN];
      load_b<TN>(b, it.ad, k, n0, l16);
      zero_past_rank<TN>(b, k);
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        if (((it.mine >> (16 * tm)) & 0xFFFF) == 0) continue;  // uniform
        v4f v[kLoraMaxParts][2];
        if ((it.mine >> (16 * tm + l16)) & 1) {
          const float* from = a.v + (uint64_t)(m0 + 16 * tm + l16) * a.parts * a.ld + k;
#pragma unroll
          for (uint32_t p = 0; p < kLoraMaxParts; ++p) {  // (the last part again past the end: not added)
            v[p][0] = *reinterpret_cast<const v4f*>(from + min(p, a.parts - 1) * a.ld);
            v[p][1] = *reinterpret_cast<const v4f*>(from + min(p, a.parts - 1) * a.ld + 4);
          }
        } else {
#pragma unroll
          for (uint32_t p = 0; p < kLoraMaxParts; ++p) v[p][0] = v[p][1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (uint32_t p = 1; p < kLoraMaxParts; ++p) {
          if (p < a.parts) {
            v[0][0] += v[p][0];
            v[0][1] += v[p][1];
          }
        }
        uint2 h0, h1, r0, r1;
        split_bf16(v[0][0], s, h0, r0);
        split_bf16(v[0][1], s, h1, r1);
        const u32x4 hi = {h0.x, h0.y, h1.x, h1.y}, lo = {r0.x, r0.y, r1.x, r1.y};
        accumulate<TN>(acc, tm, b, hi, lo, (it.mine >> (16 * tm + l16)) & 1);
      }
    }
  }

  // Few rows (decode: up to an adapter a row): the workgroup's NT threads sum,
  // scale and split v of its rows into LDS once; then its waves share the items,
  // each with the B fragments of the next one in flight.  Called by the whole
  // workgroup; LDS must be free before and is free after.  At most
  // 64 * (128 * 4 + 16) bytes of it are used.
  template <int TM, int TN, int NT, class Acc>
  __device__ __forceinline__ void add_shared(Acc&& acc, uint8_t* smem, uint32_t m0, uint32_t n0, uint32_t M,
                                             uint32_t lane, uint32_t first, uint32_t stride) const {
    const uint32_t l16 = lane & 15, q = lane >> 4;
    Items it = items<TM>(m0, M, lane, first, stride);
    if (it.left == 0) return;  // uniform over the workgroup
    u32x4 b0[TN], b1[TN];
    uint32_t k0 = 0, k1 = 0;
    uint64_t mine0 = 0, mine1 = 0;
    // the next item's loads; after the last one, loads all the same (of any
    // adapter, in bounds), so that no branch hides them from the waits
    auto load = [&](u32x4 (&b)[TN], uint32_t& k, uint64_t& mine) __attribute__((always_inline)) -> bool {
      const bool more = it.next();
      k = 32 * it.step + 8 * q;
      mine = it.mine;
      load_b<TN>(b, it.ad, k, n0, l16);
      sched_fence();
      return more;
    };
    bool more = load(b0, k0, mine0);
    // rows of `pitch` bytes: the high halves of ld values, then the low ones
    const uint32_t pitch = a.ld * 4 + 16, quads = a.ld / 4, rows = min(16u * TM, M - m0);
    for (uint32_t i = threadIdx.x; i < rows * quads; i += NT) {
      const uint32_t r = i / quads, c = i % quads, id = lora_id(a, m0 + r);
      if (id == 0xFFFFFFFFu) continue;
      const float* from = a.v + (uint64_t)(m0 + r) * a.parts * a.ld + 4 * c;
      v4f v[kLoraMaxParts];
#pragma unroll
      for (uint32_t p = 0; p < kLoraMaxParts; ++p)
        v[p] = *reinterpret_cast<const v4f*>(from + min(p, a.parts - 1) * a.ld);
#pragma unroll
      for (uint32_t p = 1; p < kLoraMaxParts; ++p)
        if (p < a.parts) v[0] += v[p];
      uint2 hi, lo;
      split_bf16(v[0], a.scale[id], hi, lo);
      *reinterpret_cast<uint2*>(smem + r * pitch + 8 * c) = hi;
      *reinterpret_cast<uint2*>(smem + r * pitch + 2 * a.ld + 8 * c) = lo;
    }
    __syncthreads();
    auto apply = [&](u32x4 (&b)[TN], uint32_t k, uint64_t mine) __attribute__((always_inline)) {
      zero_past_rank<TN>(b, k);
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        if (((mine >> (16 * tm)) & 0xFFFF) == 0) continue;  // uniform
        const bool own = (mine >> (16 * tm + l16)) & 1;
        u32x4 hi = {0, 0, 0, 0}, lo = {0, 0, 0, 0};
        if (own) {
          const uint8_t* at = smem + (16 * tm + l16) * pitch + 2 * k;
          hi = *reinterpret_cast<const u32x4*>(at);
          lo = *reinterpret_cast<const u32x4*>(at + 2 * a.ld);
        }
        accumulate<TN>(acc, tm, b, hi, lo, own);
      }
    };
    while (more) {
      more = load(b1, k1, mine1);
      apply(b0, k0, mine0);
      const bool again = load(b0, k0, mine0);
      if (!more) break;
      apply(b1, k1, mine1);
      more = again;
    }
    __syncthreads();
  }
};

}  // namespace
}  // namespace fp8q
