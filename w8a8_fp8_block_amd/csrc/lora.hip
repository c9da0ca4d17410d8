// The projection with low-rank adapters of many requests on gfx950:
//   out[m] = bf16( quant(x)[m] . W^T + scale[a] * (x[m] . A[a]^T) . B[a]^T ),
// a = ids[m], rows without an adapter the projection alone.
//
// Two parts: one pass over x quantizes it and forms v = x . A^T (fp32, in parts
// of K), and the projection's own GEMM kernels run with an epilogue that adds scale * v . B^T to
// their fp32 accumulators (lora.h), so that the sum is rounded once and out is
// written once.
#include <algorithm>

#include "gemm_pp.h"
#include "gemm_skinny.h"
#include "launch.h"
#include "lora.h"

namespace fp8q {
namespace {

// ------------------------------------------------------------------------
// Quantize and shrink, one pass over x: the FP8 codes and scales of x (the
// activation quantizer's steps) and v[m, r] = sum_k x[m, k] * A[a][r, k] in fp32
// from bf16.  A workgroup takes 16 * TM rows and one part of K, its four waves
// every fourth 128-group of it; blockIdx.z picks the rank tiles (`chunks` of NR)
// and among the rows' distinct adapters (round robin); z = 0 quantizes as well.  A lane holds values k =
// 64 h + 16 (l / 16) .. + 15, h < 2, of row l % 16 in the group, the other 96 in
// the lanes 16, 32 and 48 away: its codes are two 16-byte stores, and its
// 16-byte pieces are operands of the 16x16x32 MFMA as they stand (in an order of
// k that A's pieces share).  Per adapter every row's product is formed
// (NR rank tiles of 16) and the rows of that adapter are stored; adapters after
// a workgroup's first read its rows again, from L2.  Bound by reading A (decode:
// a few rows an adapter) or x (prompts): 25 rows of 22 adapters, rank 64, K = 5120:
// 7.7 us for 14 MB of A, a launch and two latencies; M = 1168, rank 24: 16 us; M =
// 4576, K = 17408, rank 32: 95 us for 240 MB of x and codes, 2.5 TB/s.  There 70 us remain
// without the quantization, 72 without A, and 56 with neither (2.8 TB/s: the reads of
// 32 rows 34 KB apart); more workgroups a CU (registers spill) and 64 rows a workgroup
// were slower.
// ------------------------------------------------------------------------
struct QuantOut {
  uint8_t* q;    // [M,K]
  float* rm;     // [M,K/128]
  float* km;     // [K/128,Mp]
};

// This lane's 32 values of a 128-group -> codes, the group's scale
__device__ __forceinline__ float quant_lane_group(const u32x4 (&x)[4], uint2 (&codes)[4]) {
  const uint32_t mag = 0x7FFF7FFFu;
  u16x2 mx = as_u16x2(0);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) mx = __builtin_elementwise_max(mx, as_u16x2(x[j][i] & mag));
  uint32_t amax = max((uint32_t)mx.x, (uint32_t)mx.y);
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 16));
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 32));
  const float s = group_scale(amax);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float f[8], r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf_lo(x[j][i]);
      f[2 * i + 1] = bf_hi(x[j][i]);
    }
    quotients<8>(f, s, r);
    codes[j] = make_uint2(encode4(r), encode4(r + 4));
  }
  return s;
}

template <int TM, int NR>
__global__ __launch_bounds__(256) void lora_quant_shrink_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ A, float* __restrict__ v, QuantOut out,
    const int32_t* ids, uint32_t M, uint32_t K, uint32_t Mp, uint32_t adapters, uint32_t rank, uint32_t ld,
    uint32_t parts, uint32_t chunks) {
  __shared__ v4f red[4][NR][64];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t l16 = lane & 15, q = lane >> 4;
  const uint32_t m0 = blockIdx.x * 16 * TM, part = blockIdx.y, G = K / kGroup;
  const uint32_t g0 = part * G / parts, g1 = (part + 1) * G / parts;
  const uint32_t row = m0 + lane;
  uint32_t id = 0xFFFFFFFFu;
  if (lane < 16 * TM && row < M) id = (uint32_t)ids[row];
  if (id >= adapters) id = 0xFFFFFFFFu;
  uint64_t left = __builtin_amdgcn_ballot_w64(id != 0xFFFFFFFFu);
  const uint32_t turns = gridDim.z / chunks, t0 = blockIdx.z % chunks * NR;  // this workgroup's rank tiles
  bool quantize = blockIdx.z == 0;
  const uint16_t* xr[TM];
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) xr[tm] = x + (uint64_t)min(m0 + 16 * tm + l16, M - 1) * K + 16 * q;

  // One group's rows, quantized.  The stores go through buffer resources, rows
  // past M out of range, so that no branch hides their number from the waits of
  // the loads before them.
  const __amdgpu_buffer_rsrc_t rQ = make_rsrc(out.q, M * K), rRm = make_rsrc(out.rm, M * G * 4);
  const __amdgpu_buffer_rsrc_t rKm = make_rsrc(out.km, G * Mp * 4);
  constexpr uint32_t kNoStore = 0xFFFFFF00u;  // past any bound (ceil16(M) * K < 2^32)
  auto quant = [&](uint32_t g, const u32x4 (&xf)[TM][4]) __attribute__((always_inline)) {
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      const uint32_t m = m0 + 16 * tm + l16;
      uint2 codes[4];
      const float s = quant_lane_group(xf[tm], codes);
      const uint32_t to = m < M ? m * K + g * kGroup + 16 * q : kNoStore;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{codes[2 * j].x, codes[2 * j].y, codes[2 * j + 1].x, codes[2 * j + 1].y}, rQ, to + 64 * j, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s), rRm, q == 0 && m < M ? (m * G + g) * 4 : kNoStore, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(m < M ? s : 0.0f), rKm,
                                            q == 0 && m < Mp ? (g * Mp + m) * 4 : kNoStore, 0, 0);
    }
  };
  auto load_x = [&](uint32_t g, u32x4 (&xf)[TM][4]) __attribute__((always_inline)) {
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        xf[tm][j] = *reinterpret_cast<const u32x4*>(xr[tm] + g * kGroup + 64 * (j >> 1) + 8 * (j & 1));
  };

  for (uint32_t turn = 0; left; ++turn) {
    const uint32_t ad = (uint32_t)__builtin_amdgcn_readlane((int)id, __builtin_ctzll(left));
    const uint64_t mine = __builtin_amdgcn_ballot_w64(id == ad);
    left &= ~mine;
    if (turn % turns != blockIdx.z / chunks) continue;
    const uint16_t* ar[NR];
#pragma unroll
    for (int t = 0; t < NR; ++t)
      ar[t] = A + ((uint64_t)ad * rank + min(16 * (t0 + t) + l16, rank - 1)) * K + 16 * q;
    v4f acc[TM][NR];
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)
#pragma unroll
      for (int t = 0; t < NR; ++t) acc[tm][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    // x of the next group is in flight while a group is quantized; A of the
    // group arrives (mostly from L2) under the quantization
    auto group = [&](auto quant_c, uint32_t g, const u32x4 (&xf)[TM][4], u32x4 (&xn)[TM][4])
        __attribute__((always_inline)) {
      u32x4 af[NR][4];
#pragma unroll
      for (int t = 0; t < NR; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) af[t][j] = *reinterpret_cast<const u32x4*>(ar[t] + g * kGroup + 64 * (j >> 1) + 8 * (j & 1));
      load_x(min(g + 4, g1 - 1), xn);
      sched_fence();
      if constexpr (decltype(quant_c)::value) quant(g, xf);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
#pragma unroll
          for (int t = 0; t < NR; ++t) acc[tm][t] = mfma_bf16_32(af[t][j], xf[tm][j], acc[tm][t]);
    };
    auto groups = [&](auto quant_c) __attribute__((always_inline)) {
      u32x4 xe[TM][4], xo[TM][4];
      uint32_t g = g0 + wave;
      if (g < g1) load_x(g, xe);
      while (g < g1) {
        group(quant_c, g, xe, xo);
        if ((g += 4) >= g1) break;
        group(quant_c, g, xo, xe);
        g += 4;
      }
    };
    if (quantize)
      groups(std::true_type{});
    else
      groups(std::false_type{});
    quantize = false;
    // the four waves' sums, one row tile at a time
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      const uint32_t r = 16 * tm + l16;
      if (((mine >> (16 * tm)) & 0xFFFF) == 0) continue;  // uniform over the workgroup
#pragma unroll
      for (int t = 0; t < NR; ++t) red[wave][t][lane] = acc[tm][t];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < (NR + 3) / 4; ++j) {
        const uint32_t t = 4 * j + wave, k = 16 * (t0 + t) + 4 * q;
        if (t < (uint32_t)NR && ((mine >> r) & 1) && k < ld) {
          v4f s = red[0][t][lane];
#pragma unroll
          for (int w = 1; w < 4; ++w) s += red[w][t][lane];
          if (k >= rank) s = v4f{0.0f, 0.0f, 0.0f, 0.0f};  // rank % 4 == 0
          *reinterpret_cast<v4f*>(v + ((uint64_t)(m0 + r) * parts + part) * ld + k) = s;
        }
      }
      __syncthreads();
    }
  }
  if (quantize) {  // no adapter among the rows
    for (uint32_t g = g0 + wave; g < g1; g += 4) {
      u32x4 xf[TM][4];
      load_x(g, xf);
      quant(g, xf);
    }
  }
}

// Rows up to here go in tiles of 16, their adapters dealt over workgroups; beyond, in
// tiles of 32.  32 ranks a workgroup: with all 128 in one, M = 3, K = 16128 took 31.9
// us instead of 11.1, and M = 258, K = 1792, rank 96, 48 requests 49.6 instead of
// 11.6 (there 64 ranks: 10.2; at M = 3270, K = 5760, rank 128 32 or 64 ranks: 63.5 /
// 61.7).
constexpr uint32_t kShrinkSmallM = 256;

template <int TM, int NR>
hipError_t launch_shrink_cfg(const uint16_t* x, const uint16_t* a, const LoraArgs& l, float* v,
                             const QuantOut& out, uint32_t M, uint32_t K, hipStream_t s) {
  // rank tiles up to ld, so that the zeros beyond the rank are written too
  const uint32_t tiles = (M + 16 * TM - 1) / (16 * TM), chunks = (l.ld / 16 + NR - 1) / NR;
  // one workgroup an adapter for few rows; for more, as many as leave no CU idle
  const uint32_t most = TM == 1 ? 16u : std::max(1u, std::min(8u, 512 / (tiles * l.parts * chunks)));
  const uint32_t z = std::min(std::min(most, M), l.adapters);
  lora_quant_shrink_kernel<TM, NR><<<dim3(tiles, l.parts, z * chunks), dim3(256), 0, s>>>(
      x, a, v, out, l.ids, M, K, m_pad16(M), l.adapters, l.rank, l.ld, l.parts, chunks);
  return hipGetLastError();
}

hipError_t launch_shrink(const uint16_t* x, const uint16_t* a, const LoraArgs& l, float* v,
                         const QuantOut& out, uint32_t M, uint32_t K, hipStream_t s) {
  if (M <= kShrinkSmallM) return launch_shrink_cfg<1, 2>(x, a, l, v, out, M, K, s);
  return launch_shrink_cfg<2, 2>(x, a, l, v, out, M, K, s);
}

// ------------------------------------------------------------------------
// The projection's GEMM kernels with the adapters' epilogue.
// ------------------------------------------------------------------------
struct Gemm {
  const uint8_t* a;
  const float* as;
  const uint8_t* w;
  const float* ws;
  uint16_t* out;
  uint32_t M, N, K, Mp;
};

template <int TM, int TN, int NWV, int U, bool SPLIT>
__global__ __launch_bounds__(64 * NWV) void lora_skinny_kernel(Gemm g, uint32_t base, uint32_t rem,
                                                               float* __restrict__ part, LoraArgs l) {
  gemm_skinny_body<TM, TN, NWV, U, false, SPLIT>(g.a, g.as, g.w, g.ws, g.out, g.M, g.N, g.K, g.Mp, base,
                                                 rem, part, LoraEpilogue{l});
}

template <int TM, int GW>
__global__ __launch_bounds__(512) void lora_decode_kernel(Gemm g, uint32_t base, uint32_t rem, LoraArgs l) {
  gemm_decode_body<TM, GW, false>(g.a, g.as, g.w, g.ws, g.out, g.M, g.N, g.K, g.Mp, base, rem,
                                  LoraEpilogue{l});
}

template <int STAGES, bool SPLIT>
__global__ __launch_bounds__(256, 2) void lora_tiled_kernel(Gemm g, uint32_t tiles_m, uint32_t tiles_n,
                                                         uint32_t splits, float* __restrict__ part, LoraArgs l) {
  uint32_t tmi, tni, split = 0;
  if constexpr (SPLIT)
    tile_split_coords(tiles_m, tiles_n, splits, tmi, tni, split);
  else
    tile_coords(tiles_m, tiles_n, tmi, tni);
  gemm_tiled_body<128, 128, 2, 2, STAGES, false, SPLIT>(g.a, g.as, g.w, g.ws, g.out, tmi * 128, tni * 128, g.N,
                                                        g.K, g.Mp, split, splits, part,
                                                        DenseRows{g.M, g.M}, LoraEpilogue{l});
}

__global__ __launch_bounds__(512) void lora_pp_kernel(Gemm g, uint32_t tiles_m, uint32_t tiles_n, LoraArgs l) {
  uint32_t tmi, tni;
  tile_coords(tiles_m, tiles_n, tmi, tni);
  gemm_pp_body<3, false, false>(g.a, g.as, g.w, g.ws, g.out, tmi * 256, tni * 128, g.N, g.K, g.Mp,
                                FfnArgs{nullptr, nullptr, nullptr, nullptr, 0}, DenseRows{g.M, g.M},
                                LoraEpilogue{l});
}

template <int TM, int TN, bool SPLIT>
hipError_t launch_skinny_cfg(const Gemm& g, uint32_t grid, uint32_t base, uint32_t rem, uint32_t splits,
                             float* part, const LoraArgs& l, hipStream_t s) {
  constexpr int NWV = skinny_waves(TM, TN), U = skinny_unroll(TM, TN);
  // partial sums; before them, v of the rows (64 * 528 bytes at most)
  constexpr int LDS = std::max(NWV * TN * TM * 1024, 16 * TM * (int)(kMaxLoraRank * 4 + 16));
  const hipError_t e = allow_lds<&lora_skinny_kernel<TM, TN, NWV, U, SPLIT>, LDS>();
  if (e != hipSuccess) return e;
  const uint32_t row_tiles = (g.M + 16 * TM - 1) / (16 * TM);
  lora_skinny_kernel<TM, TN, NWV, U, SPLIT>
      <<<dim3(grid, row_tiles, splits), dim3(64 * NWV), LDS, s>>>(g, base, rem, part, l);
  return hipGetLastError();
}

template <bool SPLIT>
hipError_t launch_skinny(const Gemm& g, uint32_t grid, uint32_t base, uint32_t rem, uint32_t tn, uint32_t splits,
                         float* part, const LoraArgs& l, hipStream_t s) {
#define FP8Q_LORA_TN(TM_)                                                                    \
  (tn <= 2   ? launch_skinny_cfg<TM_, 2, SPLIT>(g, grid, base, rem, splits, part, l, s)      \
   : tn <= 4 ? launch_skinny_cfg<TM_, 4, SPLIT>(g, grid, base, rem, splits, part, l, s)      \
   : tn <= 6 ? launch_skinny_cfg<TM_, 6, SPLIT>(g, grid, base, rem, splits, part, l, s)      \
             : launch_skinny_cfg<TM_, 8, SPLIT>(g, grid, base, rem, splits, part, l, s))
  switch ((g.M + 15) / 16) {
    case 1: return FP8Q_LORA_TN(1);
    case 2: return FP8Q_LORA_TN(2);
    case 3: return FP8Q_LORA_TN(3);
    default: return FP8Q_LORA_TN(4);
  }
#undef FP8Q_LORA_TN
}

template <int TM, int GW>
hipError_t launch_decode_cfg(const Gemm& g, uint32_t grid, uint32_t base, uint32_t rem, uint32_t lds,
                             const LoraArgs& l, hipStream_t s) {
  const hipError_t e = allow_lds<&lora_decode_kernel<TM, GW>, kDecodeLds>();
  if (e != hipSuccess) return e;
  lora_decode_kernel<TM, GW><<<dim3(grid), dim3(512), lds, s>>>(g, base, rem, l);
  return hipGetLastError();
}

template <int TM>
hipError_t launch_decode(const Gemm& g, uint32_t gw, uint32_t grid, uint32_t base, uint32_t rem, uint32_t lds,
                         const LoraArgs& l, hipStream_t s) {
  if (gw == 2) return launch_decode_cfg<TM, 2>(g, grid, base, rem, lds, l, s);
  if (gw == 4) return launch_decode_cfg<TM, 4>(g, grid, base, rem, lds, l, s);
  if (gw == 5) return launch_decode_cfg<TM, 5>(g, grid, base, rem, lds, l, s);
  return launch_decode_cfg<TM, 6>(g, grid, base, rem, lds, l, s);
}

template <int STAGES, bool SPLIT>
hipError_t launch_tiled(const Gemm& g, uint32_t splits, float* part, const LoraArgs& l, hipStream_t s) {
  using C = TileCfg<128, 128, 2, 2, STAGES, false>;
  static_assert(128 * (kMaxLoraRank * 4 + 16) <= C::LDS_BYTES, "the rows' v in the operand ring");
  const hipError_t e = allow_lds<&lora_tiled_kernel<STAGES, SPLIT>, C::LDS_BYTES>();
  if (e != hipSuccess) return e;
  const uint32_t tiles_m = (g.M + 127) / 128, tiles_n = g.N / 128;
  lora_tiled_kernel<STAGES, SPLIT>
      <<<dim3(tiles_m * tiles_n * splits), dim3(C::NT), C::LDS_BYTES, s>>>(g, tiles_m, tiles_n, splits, part, l);
  return hipGetLastError();
}

hipError_t launch_pp(const Gemm& g, const LoraArgs& l, hipStream_t s) {
  using C = PpCfg<3, false, false>;
  static_assert(C::BM * (kMaxLoraRank * 4 + 16) <= C::LDS_BYTES, "the rows' v in the operand ring");
  const hipError_t e = allow_lds<&lora_pp_kernel, C::LDS_BYTES>();
  if (e != hipSuccess) return e;
  const uint32_t tiles_m = (g.M + 255) / 256, tiles_n = g.N / 128;
  lora_pp_kernel<<<dim3(tiles_m * tiles_n), dim3(C::NT), C::LDS_BYTES, s>>>(g, tiles_m, tiles_n, l);
  return hipGetLastError();
}

uint32_t lora_ld(uint32_t rank) { return (rank + 31) / 32 * 32; }

// Parts of K of the shrink: as many as keep the grid within 512 workgroups (two
// a CU, one round), with at least four groups (one a wave) in each.  (Any M: the
// size query takes an empty batch and numbers no call accepts.)
uint32_t lora_parts(uint32_t M, uint32_t K) {
  const uint64_t wgs = M <= kShrinkSmallM ? (M + 15) / 16 * std::min(16u, M) : ((uint64_t)M + 31) / 32;
  const uint32_t fit = (uint32_t)(512 / std::max<uint64_t>(wgs, 1));
  return std::max(1u, std::min(std::min(kLoraMaxParts, fit), K / (4 * kGroup)));
}

}  // namespace

uint64_t lora_workspace_bytes(uint32_t M, uint32_t K, uint32_t rank) {
  return (uint64_t)M * lora_parts(M, K) * lora_ld(rank) * 4;
}

hipError_t launch_lora_quant_shrink(const uint16_t* x, const uint16_t* a, const int32_t* ids, uint8_t* x_q,
                                    float* x_s_rm, float* x_s_km, void* workspace, uint32_t M, uint32_t K,
                                    uint32_t adapters, uint32_t rank, hipStream_t s) {
  LoraArgs l{};
  l.ids = ids;
  l.adapters = adapters;
  l.rank = rank;
  l.ld = lora_ld(rank);
  l.parts = lora_parts(M, K);
  float* v = static_cast<float*>(workspace);
  const QuantOut out{x_q, x_s_rm, x_s_km};
  return launch_shrink(x, a, l, v, out, M, K, s);
}

hipError_t launch_lora_gemm(const uint8_t* a, const float* a_s_km, const uint8_t* w, const float* w_s,
                            uint16_t* out, const void* workspace, float* part, const uint16_t* lora_b,
                            const float* lora_scale, const int32_t* ids, uint32_t M, uint32_t N, uint32_t K,
                            uint32_t adapters, uint32_t rank, uint32_t cus, int kernel, uint32_t splits,
                            hipStream_t s) {
  const Gemm g{a, a_s_km, w, w_s, out, M, N, K, m_pad16(M)};
  const LoraArgs l{static_cast<const float*>(workspace), lora_b, lora_scale, ids, adapters, rank, lora_ld(rank),
                   lora_parts(M, K), N};
  if (splits >= 2) {
    hipError_t e;
    const uint32_t grid = skinny_split_grid(N, splits, cus);
    const uint32_t cols = skinny_split_columns(N, splits, cus);
    if (M <= 64 && cols <= 128)
      e = launch_skinny<true>(g, grid, N / 4 / grid, N / 4 % grid, (cols + 15) / 16, splits, part, l, s);
    else if ((uint64_t)((M + 127) / 128) * (N / 128) * splits <= cus)
      e = launch_tiled<3, true>(g, splits, part, l, s);
    else
      e = launch_tiled<2, true>(g, splits, part, l, s);
    return e != hipSuccess ? e : launch_splitk_reduce(part, out, M, N, splits, s);
  }
  if (kernel == 2) {
    uint32_t grid = 0, base = 0, rem = 0, tn = 0, tm = 0, gw = 0, lds = 0;
    skinny_grid(M, N, cus, grid, base, rem, tn);
    if (decode_plan(M, K, base, rem, tm, gw, lds))
      return tm == 1 ? launch_decode<1>(g, gw, grid, base, rem, lds, l, s)
                     : launch_decode<2>(g, gw, grid, base, rem, lds, l, s);
    return launch_skinny<false>(g, grid, base, rem, tn, 1, nullptr, l, s);
  }
  if (kernel == 1) return launch_tiled<2, false>(g, 1, nullptr, l, s);
  return launch_pp(g, l, s);
}

}  // namespace fp8q
