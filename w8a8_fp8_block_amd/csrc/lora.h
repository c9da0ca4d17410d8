// Low-rank adapters beside a shared projection: the epilogue that adds a row's
// adapter to the GEMM's fp32 accumulators (lora.hip holds the kernels).
#pragma once

#include "mfma_common.h"

namespace fp8q {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// v = x . A^T in kLoraParts contiguous parts of K at most, [M][parts][ld] fp32
// (ld: the rank rounded up to 32, zero beyond it).
constexpr uint32_t kLoraMaxParts = 8;

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

// out[m, n] += scale[a] * sum_r v[m, r] * B[a][n, r] for the rows m of adapter
// a, on the GEMM's accumulator layout (lane l: row l % 16 of its 16-row tile,
// columns 4 * (l / 16) .. +3).  A wave walks the distinct adapters of its rows
// (up to 64, a row a lane); for each, one pass over the rank in MFMA steps of 32
// with the other rows' v zeroed.  The scaled v enters the bf16 product as the
// sum of two bf16 numbers (its rounding and the rest), so that the delta keeps
// about 16 bits of v, and the accumulator is rounded once, with the base.
// The adapters are dealt over `stride` participants, `first` this one's index.
struct LoraEpilogue {
  LoraArgs a;
  template <int TM, int TN, class Acc>
  __device__ __forceinline__ void add(Acc&& acc, uint32_t m0, uint32_t n0, uint32_t M, uint32_t lane,
                                      uint32_t first, uint32_t stride, uint32_t split) const {
    static_assert(TM <= 4, "a row a lane");
    if (split != 0) return;  // tiled split-K: the first part adds
    const uint32_t l16 = lane & 15, q = lane >> 4;
    const uint32_t row = m0 + lane;
    const uint32_t id = lane < 16 * TM && row < M ? lora_id(a, row) : 0xFFFFFFFFu;
    uint64_t left = __builtin_amdgcn_ballot_w64(id != 0xFFFFFFFFu);
    for (uint32_t turn = 0; left; ++turn) {
      const uint32_t ad = (uint32_t)__builtin_amdgcn_readlane((int)id, __builtin_ctzll(left));
      const uint64_t mine = __builtin_amdgcn_ballot_w64(id == ad);
      left &= ~mine;
      if (turn % stride != first) continue;
      const float s = a.scale[ad];
      const uint16_t* b = a.b + (uint64_t)ad * a.N * a.rank;
      for (uint32_t k0 = 0; k0 < a.rank; k0 += 32) {
        const uint32_t k = k0 + 8 * q;
        u32x4 bf[TN];
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          // past the rank or the columns: any in-bounds values, zeroed or unused
          bf[t] = *reinterpret_cast<const u32x4*>(b + (uint64_t)min(n0 + 16 * t + l16, a.N - 1) * a.rank +
                                                  min(k, a.rank - 8));
          if (k >= a.rank) bf[t] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
          if (((mine >> (16 * tm)) & 0xFFFF) == 0) continue;  // uniform
          const bool on = (mine >> (16 * tm + l16)) & 1;
          u32x4 hi = {0, 0, 0, 0}, lo = {0, 0, 0, 0};
          if (on) {
            const float* v = a.v + (uint64_t)(m0 + 16 * tm + l16) * a.parts * a.ld + k;
            v4f v0 = {0, 0, 0, 0}, v1 = {0, 0, 0, 0};
            for (uint32_t p = 0; p < a.parts; ++p) {
              v0 += *reinterpret_cast<const v4f*>(v + p * a.ld);
              v1 += *reinterpret_cast<const v4f*>(v + p * a.ld + 4);
            }
            v0 *= s;
            v1 *= s;
            uint32_t h[8], r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float f = i < 4 ? v0[i] : v1[i - 4];
              h[i] = bf16_rne(f);
              r[i] = bf16_rne(f - __uint_as_float(h[i] << 16));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              hi[i] = h[2 * i] | (h[2 * i + 1] << 16);
              lo[i] = r[2 * i] | (r[2 * i + 1] << 16);
            }
          }
#pragma unroll
          for (int t = 0; t < TN; ++t) {
            acc(tm, t) = mfma_bf16_32(bf[t], lo, acc(tm, t));
            acc(tm, t) = mfma_bf16_32(bf[t], hi, acc(tm, t));
          }
        }
      }
    }
  }
};

}  // namespace
}  // namespace fp8q
