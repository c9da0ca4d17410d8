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

// v * s as the sum of two bf16 numbers (its rounding and the rest), four at a time.
// The first is held to bf16's range: what lies beyond, up to an infinity or a NaN,
// is the rest's (an infinity's own rest would be inf - inf).
__device__ __forceinline__ void split_bf16(const v4f& v, float s, uint2& hi, uint2& lo) {
#pragma clang fp contract(off)  // one f for both terms
  typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
  constexpr float kMost = 0x1.FEp127f;  // bf16's largest
  v4f f, c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = v[i] * s;
    c[i] = __builtin_amdgcn_fmed3f(f[i], -kMost, kMost);
  }
  const v4bf h = __builtin_convertvector(c, v4bf);
  hi = __builtin_bit_cast(uint2, h);
  lo = __builtin_bit_cast(uint2, __builtin_convertvector(f - __builtin_convertvector(h, v4f), v4bf));
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
// 13 us beside the base's 26); at prompts by the latency of its steps: M = 1168, N =
// 6144, K = 5120, rank 24, 19 requests: 47 us, of which the dense GEMM is about 39, and
// 51 where v was read from global memory at each adapter's steps; M = 278, N = 12032,
// rank 88, 54 requests: the whole call 60 against 121 (54 of 4 adapters, 87 of 23).
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

  // v of `rows` rows from m0 on, summed over its parts, scaled and split, into LDS
  // by the workgroup's NT threads: rows of pitch() bytes, the high halves of ld
  // values, then the low ones.  (Rows without an adapter: unused values.)
  __device__ __forceinline__ uint32_t pitch() const { return a.ld * 4 + 16; }
  template <int NT>
  __device__ __forceinline__ void stage(uint8_t* smem, uint32_t m0, uint32_t rows) const {
    const uint32_t quads = a.ld / 4;
#pragma unroll 2
    for (uint32_t i = threadIdx.x; i < rows * quads; i += NT) {
      const uint32_t r = i / quads, c = i % quads;
      const float* from = a.v + (uint64_t)(m0 + r) * a.parts * a.ld + 4 * c;
      v4f v[kLoraMaxParts];
#pragma unroll
      for (uint32_t p = 0; p < kLoraMaxParts; ++p)  // (the last part again past the end: not added)
        v[p] = *reinterpret_cast<const v4f*>(from + min(p, a.parts - 1) * a.ld);
      const float s = a.scale[min((uint32_t)a.ids[m0 + r], a.adapters - 1)];
#pragma unroll
      for (uint32_t p = 1; p < kLoraMaxParts; ++p)
        if (p < a.parts) v[0] += v[p];
      uint2 hi, lo;
      split_bf16(v[0], s, hi, lo);
      *reinterpret_cast<uint2*>(smem + r * pitch() + 8 * c) = hi;
      *reinterpret_cast<uint2*>(smem + r * pitch() + 2 * a.ld + 8 * c) = lo;
    }
  }

  // One item's B fragments and what it applies to
  template <int TN>
  struct Fetched {
    u32x4 b[TN];
    uint32_t k;
    uint64_t mine;
  };
  // The next item's loads; after the last one, loads all the same (of any adapter,
  // in bounds), so that no branch hides them from the waits.
  template <int TN>
  __device__ __forceinline__ bool fetch(Items& it, Fetched<TN>& f, uint32_t n0, uint32_t l16, uint32_t q) const {
    const bool more = it.next();
    f.k = 32 * it.step + 8 * q;
    f.mine = it.mine;
    load_b<TN>(f.b, it.ad, f.k, n0, l16);
    sched_fence();
    return more;
  }
  // f applied to the wave's rows, whose v starts at `v` in LDS
  template <int TM, int TN, class Acc>
  __device__ __forceinline__ void apply(Acc&& acc, Fetched<TN>& f, const uint8_t* v, uint32_t l16) const {
    zero_past_rank<TN>(f.b, f.k);
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      if (((f.mine >> (16 * tm)) & 0xFFFF) == 0) continue;  // uniform
      const bool own = (f.mine >> (16 * tm + l16)) & 1;
      u32x4 hi = {0, 0, 0, 0}, lo = {0, 0, 0, 0};
      if (own) {
        const uint8_t* at = v + (16 * tm + l16) * pitch() + 2 * f.k;
        hi = *reinterpret_cast<const u32x4*>(at);
        lo = *reinterpret_cast<const u32x4*>(at + 2 * a.ld);
      }
      accumulate<TN>(acc, tm, f.b, hi, lo, own);
    }
  }
  // All items from the one in f0 on, each with the next one's B in flight
  template <int TM, int TN, class Acc>
  __device__ __forceinline__ void apply_all(Acc&& acc, Items& it, Fetched<TN>& f0, bool more, const uint8_t* v,
                                            uint32_t n0, uint32_t l16, uint32_t q) const {
    Fetched<TN> f1;
    while (more) {
      more = fetch<TN>(it, f1, n0, l16, q);
      apply<TM, TN>(acc, f0, v, l16);
      const bool again = fetch<TN>(it, f0, n0, l16, q);
      if (!more) break;
      apply<TM, TN>(acc, f1, v, l16);
      more = again;
    }
  }

  // Tiled kernels: the workgroup stages v of its BM rows, where the operand ring
  // was (BM * (128 * 4 + 16) bytes at most); then each wave takes the adapters of
  // its own rows, band .. band + 16 * TM.
  template <int TM, int TN, int NT, int BM, class Acc>
  __device__ __forceinline__ void add(Acc&& acc, uint8_t* smem, uint32_t m0, uint32_t band, uint32_t n0, uint32_t M,
                                      uint32_t lane, uint32_t split) const {
    if (split != 0) return;  // split-K: the first part adds
    const uint32_t l16 = lane & 15, q = lane >> 4;
    Items it = items<TM>(m0 + band, M, lane, 0, 1);
    Fetched<TN> f;
    const bool more = fetch<TN>(it, f, n0, l16, q);
    __syncthreads();  // every wave is done with the ring
    stage<NT>(smem, m0, min((uint32_t)BM, M - m0));
    __syncthreads();
    apply_all<TM, TN>(acc, it, f, more, smem + band * pitch(), n0, l16, q);
  }

  // Decode widths (up to an adapter a row): the waves hold the same rows and
  // share the items.  LDS must be free before and is free after; at most 64 *
  // (128 * 4 + 16) bytes of it are used.
  template <int TM, int TN, int NT, class Acc>
  __device__ __forceinline__ void add_shared(Acc&& acc, uint8_t* smem, uint32_t m0, uint32_t n0, uint32_t M,
                                             uint32_t lane, uint32_t first, uint32_t stride) const {
    const uint32_t l16 = lane & 15, q = lane >> 4;
    Items it = items<TM>(m0, M, lane, first, stride);
    if (it.left == 0) return;  // uniform over the workgroup
    Fetched<TN> f;
    const bool more = fetch<TN>(it, f, n0, l16, q);
    stage<NT>(smem, m0, min(16u * TM, M - m0));
    __syncthreads();
    apply_all<TM, TN>(acc, it, f, more, smem, n0, l16, q);
    __syncthreads();
  }
};

}  // namespace
}  // namespace fp8q
