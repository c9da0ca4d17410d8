// Products grouped by expert on gfx950 (block-scaled FP8):
//   out[p, n] = bf16( sum_kb a_s[kb][r] * w_s[e][n/128][kb] * P(r, e, n, kb) ),
//   r = order[p] / per_row (or p), e: offsets[e] <= p < offsets[e + 1],
// with P the 128-deep e4m3 dot products of the dense GEMM (gemm.hip).
#include <algorithm>

#include "group_pp.h"
#include "launch.h"

namespace fp8q {
namespace {

// Up to two weight sets that read the same rows (gate and up): blockIdx.y picks.
struct GroupWeights {
  const uint8_t* w[2];
  const float* ws[2];
  uint16_t* out[2];
};

// ------------------------------------------------------------------------
// Streaming kernel for experts of few rows.  The product is then bound by
// reading each active expert's weights once from HBM, so the design keeps a
// steady stream of weight loads on every CU: one persistent workgroup of eight
// waves per CU takes an equal, contiguous run of units (a unit: 16 * CW columns
// of one expert's row tile over all of K) and runs them as one pipeline, the
// loads of the next unit following the last of the current one without a gap.
//
// A stage is 16 KB of weights: KS = 8 / CW consecutive K blocks of 16 * CW
// columns.  Wave (cw, kw) loads and multiplies its own 16 columns x K block kw
// of every stage; the stage's activations (16 * TM rows x KS blocks), shared by
// the waves, and each wave's scales come with it, all by direct loads into a
// ring of ST slots with one barrier a stage.  Rows past the group and K blocks
// past K are out-of-range loads: zeros without a memory access.  At a unit's end
// the KS partial tiles are added in K order through LDS.
//
// 25 tokens of 64 experts, top 8, N = 2048, K = 5120: 97 us for 599 MB, 6.2 TB/s (each
// weight read once by the counters; 7.0 is the rate of the loads alone), 115 us for
// gate and up (664 MB) of 16 tokens, top 6, H = 5120, I = 1408.  One token, 4 experts,
// N = 2048, K = 1024: 6.7 us, the latency of one fill of the pipeline.
// ------------------------------------------------------------------------
constexpr int kOffsetsLds = (kMaxExperts + 1) * 4;
template <int TM, int TN, int CW, int KS>
struct StreamCfg {
  static constexpr int NW = CW * KS, BN = 16 * TN * CW;
  static constexpr int W_BYTES = NW * TN * 2048;               // weights of a stage
  static constexpr int A_BYTES = KS * TM * 2048;               // activations of a stage
  static constexpr int SA = (TM + 3) / 4;                      // 64-row loads of the row scales
  static constexpr int SC_BYTES = SA * 256 + 256;              // per K block: row scales, the waves' weight scales
  static constexpr int SLOT = W_BYTES + A_BYTES + KS * SC_BYTES;
  // besides its weights a wave loads JOBS of its K block's 1 KB activation
  // pieces, row scales and weight scales (dealt over the CW waves)
  static constexpr int JOBS = (2 * TM + SA + 1 + CW - 1) / CW;
  static constexpr int LOADS = 2 * TN + JOBS;                  // loads a wave and stage
  static constexpr int RED = (NW - CW) * TM * TN * 1024;       // partial tiles of the waves with kw > 0
  static constexpr int SPARE = 256;                            // where loads without a job go
  static constexpr int ROOM = (160 * 1024 - kOffsetsLds - RED - SPARE) / SLOT, ST = ROOM < 8 ? ROOM : 8;
  static constexpr int OFFSETS = ST * SLOT + RED + SPARE, LDS = OFFSETS + kOffsetsLds;
  static_assert(ST >= 3 && (ST - 2) * LOADS < 63, "pipeline");
};
constexpr uint32_t kWholeWorkers = 4;
// past any operand's bound (ceil16(rows) * K < 2^32, so at most 0xFFFFF800)
constexpr uint32_t kOutOfRange = 0xFFFFFF00u;

// Position of a worker in its run of granules (16 * TN columns of a row tile):
// the current unit is `width` <= CW granules from `col` on.
struct UnitCursor {
  uint32_t expert, m0, end, set, col, width, left;  // left: the worker's granules from col on
  // size of the unit at col: the worker's part of this row tile in equal units
  template <int CW>
  __device__ __forceinline__ void size(uint32_t granules) {
    const uint32_t seg = min(granules - col, left), n = (seg + CW - 1) / CW;
    width = n ? (seg + n - 1) / n : 0;
  }
  // the next unit (left = 0: none); true if its rows differ
  template <int BM, int CW>
  __device__ __forceinline__ bool next(const uint32_t* offsets, uint32_t sets, uint32_t granules) {
    col += width;
    left -= width;
    bool moved = false;
    if (col == granules && left > 0) {
      col = 0;
      if (++set == sets) {
        set = 0;
        moved = true;
        m0 += BM;
        while (m0 >= end) {  // (granules are left: an expert with rows follows)
          ++expert;
          m0 = __builtin_amdgcn_readfirstlane(offsets[expert]);
          end = __builtin_amdgcn_readfirstlane(offsets[expert + 1]);
        }
      }
    }
    size<CW>(granules);
    return moved;
  }
};

// e4m3 codes -> f16, exactly: 8 of a lane's 32 codes of a K block (step s of 4)
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
__device__ __forceinline__ v8h codes_f16(const v8i& c, int s) {
  v8h h;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)c[2 * s + i], 1.0f, false);
    const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)c[2 * s + i], 1.0f, true);
    h[4 * i] = a[0];
    h[4 * i + 1] = a[1];
    h[4 * i + 2] = b[0];
    h[4 * i + 3] = b[1];
  }
  return h;
}

// F16: the products of a K block by f16 MFMAs on the widened codes.  The FP8
// MFMA's 128-deep sums are off by 1.4e-5 of their RMS (its products are summed
// to about 16 bits; the same for the 32-deep form), the f16 one's by 1e-8.
// Where the result is rounded to bf16 and quantized again, as gate and up are,
// that moves values across rounding boundaries: 16 tokens of 64 experts, H = 5120, I
// = 1408, gave an expert FFN 3.7e-3 of its norm from the 64-bit value, against
// 2.4e-3 with f16, the bf16 roundings of the experts' outputs and of their sum.  The conversions and the
// slower MFMA hide under the weight stream.
template <int TM, int TN, int CW, int KS, bool F16>
__global__ __launch_bounds__(64 * CW * KS) void group_stream_kernel(const uint8_t* __restrict__ A,
                                                           const float* __restrict__ As, GroupWeights gw,
                                                           uint32_t sets, Groups g, uint32_t N, uint32_t K,
                                                           uint32_t Mp) {
  using C = StreamCfg<TM, TN, CW, KS>;
  constexpr int BM = 16 * TM, ST = C::ST;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t cw = wave % CW, kw = wave / CW;
  const uint32_t l16 = lane & 15, q = lane >> 4;
  const uint32_t G = K / kGroup, stages = (G + KS - 1) / KS, granules = N / (16 * TN);

  // this worker's granules; workers are numbered XCD by XCD
  RowTiles<BM> rt(g, lane);
  const uint32_t workers = gridDim.x, bid = blockIdx.x;
  const uint32_t w = workers % 8 == 0 ? (bid & 7) * (workers / 8) + (bid >> 3) : bid;
  // Few row tiles: each gets whole workers, so that no worker crosses from one
  // to the next (a crossing adds a unit, and a stage takes nearly the same time
  // however wide).  Many: equal runs.
  const uint32_t each = sets * granules;  // granules of a row tile
  if (rt.total == 0) return;
  uint32_t tile, col, count;
  if (rt.total * kWholeWorkers <= workers) {
    tile = w * rt.total / workers;
    const uint32_t first = (tile * workers + rt.total - 1) / rt.total;
    const uint32_t n = ((tile + 1) * workers + rt.total - 1) / rt.total - first;
    col = (w - first) * each / n;
    count = (w - first + 1) * each / n - col;
  } else {
    const uint64_t all = (uint64_t)rt.total * each;
    const uint64_t g0 = all * w / workers, g1 = all * (w + 1) / workers;
    tile = (uint32_t)(g0 / each);
    col = (uint32_t)(g0 % each);
    count = (uint32_t)(g1 - g0);
  }
  if (count == 0) return;  // uniform over the workgroup
  UnitCursor ld;
  {
    uint32_t row0, prior;
    rt.find(g, tile, 1, ld.expert, row0, ld.end, prior);
    ld.m0 = row0 + (tile - prior) * BM;
    ld.set = col / granules;
    ld.col = col % granules;
    ld.left = count;
    ld.size<CW>(granules);
  }
  UnitCursor cu = ld;
  uint32_t* offs = reinterpret_cast<uint32_t*>(smem + C::OFFSETS);
  for (uint32_t e = threadIdx.x; e <= g.E; e += 64 * C::NW) offs[e] = min((uint32_t)g.offsets[e], g.R);
  __syncthreads();

  // ---- load side ----
  const __amdgpu_buffer_rsrc_t rA = make_rsrc(A, g.a_rows * K);
  const __amdgpu_buffer_rsrc_t rS = make_rsrc(As, G * Mp * 4);
  __amdgpu_buffer_rsrc_t rW, rWs;
  uint32_t w_off[2 * TN], j_off[C::JOBS];  // source offsets of this lane: weights, jobs
#pragma unroll
  for (int j = 0; j < 2 * TN; ++j) {
    const uint32_t row = 8 * j + (lane >> 3);
    w_off[j] = row * K + ((lane & 7) ^ swz(row)) * 16;
  }
  auto rows_of = [&]() __attribute__((always_inline)) {
    const GroupRows rows{g.a_rows, ld.end, g.order, g.per_row};
#pragma unroll
    for (int j = 0; j < C::JOBS; ++j) {
      const uint32_t job = cw * C::JOBS + j;
      if (job < 2 * TM) {
        const uint32_t r = job * 8 + (lane >> 3), m = ld.m0 + r;
        j_off[j] = m < ld.end ? rows.src(m) * K + ((lane & 7) ^ swz(r)) * 16 : kOutOfRange;
      } else if (job < 2 * TM + C::SA) {
        j_off[j] = rows.src(min(ld.m0 + (job - 2 * TM) * 64 + lane, ld.end - 1)) * 4;
      }
    }
  };
  auto weights_of = [&]() __attribute__((always_inline)) {
    const uint32_t n0 = (ld.col + min(cw, ld.width - 1)) * 16 * TN;  // (waves past the unit load nothing)
    rW = make_rsrc(gw.w[ld.set] + ((uint64_t)ld.expert * N + n0) * K, 16 * TN * K);
    rWs = make_rsrc(gw.ws[ld.set] + (uint64_t)ld.expert * (N / kGroup) * G, (N / kGroup) * G * 4);
#pragma unroll
    for (int j = 0; j < C::JOBS; ++j)  // lane w: the weight scale of wave w's columns
      if (cw * C::JOBS + j == 2 * TM + C::SA)
        j_off[j] = lane < CW ? (ld.col + min(lane, ld.width - 1)) * 16 * TN / kGroup * G * 4 : kOutOfRange;
  };
  rows_of();
  weights_of();
  uint32_t l_kb = kw, l_slot = 0;  // l_kb: this wave's K block of the stage to load
  const uint32_t lds0 = lds_addr(smem);
  auto issue = [&]() __attribute__((always_inline)) {
    const bool in = ld.left > 0 && l_kb < G;
    const uint32_t off = in ? 0 : kOutOfRange, k = in ? l_kb : 0, w_out = cw < ld.width ? off : kOutOfRange;
    const uint32_t slot = lds0 + l_slot * C::SLOT;
#pragma unroll
    for (int j = 0; j < 2 * TN; ++j)
      dma16_at_aux<kStreamOnce>(rW, w_off[j] | w_out, k * kGroup, slot + wave * TN * 2048 + j * 1024);
    const uint32_t a_at = slot + C::W_BYTES + kw * TM * 2048;
    const uint32_t sc_at = slot + C::W_BYTES + C::A_BYTES + kw * C::SC_BYTES;
#pragma unroll
    for (int j = 0; j < C::JOBS; ++j) {
      const uint32_t job = cw * C::JOBS + j;  // uniform over the wave
      if (job < 2 * TM)
        dma16_at(rA, j_off[j] | off, k * kGroup, a_at + job * 1024);
      else if (job < 2 * TM + C::SA)
        dma4_at(rS, j_off[j], k * Mp * 4, sc_at + (job - 2 * TM) * 256);
      else if (job == 2 * TM + C::SA)
        dma4_at(rWs, j_off[j], k * 4, sc_at + C::SA * 256);
      else
        dma4_at(rWs, kOutOfRange, 0, lds0 + ST * C::SLOT + C::RED);  // no job: keeps the count of loads
    }
    l_slot = l_slot + 1 == ST ? 0 : l_slot + 1;
    l_kb += KS;
    if (l_kb - kw >= stages * KS && ld.left > 0) {  // uniform: the unit's last stage was loaded
      l_kb = kw;
      if (ld.next<BM, CW>(offs, sets, granules)) rows_of();
      if (ld.left > 0) weights_of();
    }
  };

  // ---- compute side ----
  v4f acc[TM][TN];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)
#pragma unroll
      for (int t = 0; t < TN; ++t) acc[tm][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  };
  clear();
  const uint32_t c0 = 2 * q;
  const uint32_t lo0 = l16 * 128 + ((c0 ^ swz(l16)) * 16), lo1 = l16 * 128 + (((c0 + 1) ^ swz(l16)) * 16);
  auto frag = [&](const uint8_t* p) __attribute__((always_inline)) -> v8i {
    return join(*reinterpret_cast<const u32x4*>(p + lo0), *reinterpret_cast<const u32x4*>(p + lo1));
  };
  auto epilogue = [&]() __attribute__((always_inline)) {
    v4f* red = reinterpret_cast<v4f*>(smem + ST * C::SLOT) + lane;
    if constexpr (KS > 1) {
      if (kw > 0) {
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
#pragma unroll
          for (int t = 0; t < TN; ++t) red[(((wave - CW) * TM + tm) * TN + t) * 64] = acc[tm][t];
      }
      wait_lgkm0();
      wg_barrier();
    }
    if (kw == 0 && cw < cu.width) {
      uint16_t* out = gw.out[cu.set];
      const uint32_t n = (cu.col + cw) * 16 * TN + 4 * q;
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        const uint32_t m = cu.m0 + 16 * tm + l16;
#pragma unroll
        for (int t = 0; t < TN; ++t) {
#pragma unroll
          for (int k = 1; k < KS; ++k) acc[tm][t] += red[((((k - 1) * CW + cw) * TM + tm) * TN + t) * 64];
          if (m < cu.end) *reinterpret_cast<uint2*>(out + (uint64_t)m * N + n + 16 * t) = pack_bf16x4(acc[tm][t]);
        }
      }
    }
    clear();
  };

#pragma unroll 1
  for (int s = 0; s < ST - 1; ++s) issue();
  uint32_t slot = 0;
  while (true) {
#pragma unroll 1
    for (uint32_t s = 0; s < stages; ++s) {
      wait_vmcnt<(ST - 2) * C::LOADS>();  // own part of this stage
      wg_barrier();                       // everyone's; and the slot before is free
      issue();
      const uint8_t* p = smem + slot * C::SLOT;
      const uint8_t* sc = p + C::W_BYTES + C::A_BYTES + kw * C::SC_BYTES;
      v8i wf[TN], af[TM];
      float as[TM];
#pragma unroll
      for (int t = 0; t < TN; ++t) wf[t] = frag(p + (wave * TN + t) * 2048);
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        af[tm] = frag(p + C::W_BYTES + (kw * TM + tm) * 2048);
        as[tm] = *reinterpret_cast<const float*>(sc + (16 * tm + l16) * 4);
      }
      const float ws = *reinterpret_cast<const float*>(sc + C::SA * 256 + cw * 4);
      v4f r[TM][TN];
#pragma unroll
      for (int tm = 0; tm < TM; ++tm)
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          if constexpr (F16) {
            r[tm][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              r[tm][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(wf[t], i), codes_f16(af[tm], i), r[tm][t],
                                                                0, 0, 0);
          } else {
            r[tm][t] = mfma_e4m3_128(wf[t], af[tm]);
          }
        }
#pragma unroll
      for (int tm = 0; tm < TM; ++tm)
#pragma unroll
        for (int t = 0; t < TN; ++t) acc[tm][t] += r[tm][t] * (as[tm] * ws);
      wait_lgkm0();  // this stage's reads are done: the barrier frees its slot
      slot = slot + 1 == ST ? 0 : slot + 1;
    }
    epilogue();
    cu.next<BM, CW>(offs, sets, granules);
    if (cu.left == 0) break;
  }
  wait_vmcnt<0>();  // no direct load may still be writing LDS at exit
}

template <int TM, int TN, int CW, int KS, bool F16>
hipError_t launch_stream(const uint8_t* a, const float* as, const GroupWeights& gw, uint32_t sets,
                         const Groups& g, uint32_t N, uint32_t K, uint32_t cus, hipStream_t s) {
  using C = StreamCfg<TM, TN, CW, KS>;
  const hipError_t e = allow_lds<&group_stream_kernel<TM, TN, CW, KS, F16>, C::LDS>();
  if (e != hipSuccess) return e;
  const uint64_t units = (uint64_t)max_row_tiles(g.R, g.E, 16 * TM) * sets * (N / (16 * TN));
  const uint32_t grid = (uint32_t)(units < cus ? units : cus);
  group_stream_kernel<TM, TN, CW, KS, F16>
      <<<dim3(grid), dim3(64 * C::NW), C::LDS, s>>>(a, as, gw, sets, g, N, K, m_pad16(g.a_rows));
  return hipGetLastError();
}

// ------------------------------------------------------------------------
// The dense GEMM's tiled kernel over the experts' rows: for few tiles, for shapes
// the persistent kernel does not take (K < 512, more than 256 experts), and for
// gate and up at once.
// ------------------------------------------------------------------------
template <int BM, int BN, int WGM, int WGN, int STAGES, int WAUX>
__global__ __launch_bounds__(64 * WGM * WGN) void group_tiled_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ As, GroupWeights gw, Groups g,
    uint32_t N, uint32_t K, uint32_t Mp, uint32_t tiles_n) {
  GroupTile t;
  if (!group_tile<BM>(g, tiles_n, blockIdx.x, threadIdx.x & 63, t)) return;
  const uint32_t which = blockIdx.y;
  gemm_tiled_body<BM, BN, WGM, WGN, STAGES, false, false, GroupRows, NoEpilogue, WAUX>(
      A, As, gw.w[which] + (uint64_t)t.expert * N * K,
      gw.ws[which] + (uint64_t)t.expert * (N / kGroup) * (K / kGroup), gw.out[which], t.m0, t.tn * BN,
      N, K, Mp, 0, 1, nullptr, GroupRows{g.a_rows, t.end, g.order, g.per_row}, NoEpilogue{});
}

// Fused gate/up of the experts' FFN for shapes the persistent kernel does not take:
// the ping-pong kernel's FFN mode, 128 sorted rows by 128 intermediate columns,
// writing the quantized intermediate.  T = 4576, top 4, 32 experts, H = 5120, I =
// 2048: 515 us against the persistent kernel's 470.
__global__ __launch_bounds__(512) void group_gate_up_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ As, GroupWeights gw, Groups g,
    uint8_t* __restrict__ hq, float* __restrict__ hs, uint32_t I, uint32_t H, uint32_t Mp,
    uint32_t Mp_h, uint32_t tiles_n) {
  using C = PpCfg<3, false, true>;
  GroupTile t;
  if (!group_tile<C::BM>(g, tiles_n, blockIdx.x, threadIdx.x & 63, t)) return;
  const uint64_t wo = (uint64_t)t.expert * I * H, so = (uint64_t)t.expert * (I / kGroup) * (H / kGroup);
  gemm_pp_body<3, false, true>(
      A, As, gw.w[0] + wo, gw.ws[0] + so, nullptr, t.m0, t.tn * kGroup, I, H, Mp,
      FfnArgs{gw.w[1] + wo, gw.ws[1] + so, hq, hs, Mp_h}, GroupRows{g.a_rows, t.end, g.order, g.per_row},
      NoEpilogue{});
}

// WAUX: the weights' cache policy.  With one row tile an expert they are read
// once; with several the tiles share them through L2.
template <int WAUX>
hipError_t launch_group_128(const uint8_t* a, const float* as, const GroupWeights& gw, uint32_t sets,
                            const Groups& g, uint32_t N, uint32_t K, hipStream_t s) {
  using C = TileCfg<128, 128, 2, 2, 2, false>;
  const hipError_t e = allow_lds<&group_tiled_kernel<128, 128, 2, 2, 2, WAUX>, C::LDS_BYTES>();
  if (e != hipSuccess) return e;
  const uint32_t tiles_n = N / 128;
  group_tiled_kernel<128, 128, 2, 2, 2, WAUX><<<dim3(max_row_tiles(g.R, g.E, 128) * tiles_n, sets), dim3(C::NT),
                                          C::LDS_BYTES, s>>>(a, as, gw, g, N, K, m_pad16(g.a_rows), tiles_n);
  return hipGetLastError();
}

template <int WAUX>
hipError_t launch_group_persist(const uint8_t* a, const float* as, const GroupWeights& gw, const Groups& g,
                                uint32_t N, uint32_t K, uint32_t cus, hipStream_t s) {
  const hipError_t e = allow_lds<&group_persist_kernel<WAUX>, PersistCfg::LDS>();
  if (e != hipSuccess) return e;
  const uint32_t tiles_n = (N + 255) / 256;
  const uint64_t most = (uint64_t)max_row_tiles(g.R, g.E, 128) * tiles_n;
  group_persist_kernel<WAUX><<<dim3((uint32_t)(most < cus ? most : cus)), dim3(512), PersistCfg::LDS, s>>>(
      a, as, gw.w[0], gw.ws[0], gw.out[0], g, N, K, m_pad16(g.a_rows), tiles_n);
  return hipGetLastError();
}

// Weights bypass the caches below this mean of rows an expert.
constexpr uint32_t kReadOnceRows = 64;
// Kernel ids of the grouped product
constexpr int kGroupStream = 1, kGroupTiled = 2, kGroupPp = 3;

// By the mean rows an expert and the tiles (us).
//  Streaming below kTileMinRows; and below kFewTilesMaxRows where 128-column tiles
//  would not give every CU one.  Against the persistent kernel at E = 32, N x K =
//  2048 x 5120 and 5120 x 2048, mean 12: 54.3 / 54.3 against 62.3 / 63.3, 16: 71.2
//  / 60.7 against 62.0 / 66.0, 24: 70.5 / 72.9 against 63.9 / 66.5.  Against 128 x
//  128 tiles at E = 8, N x K = 2048 x 2048, mean 32: 13.5 / 18.1, 56: 17.4 / 18.6,
//  72: 21.8 / 15.5.
//  128 x 128 tiles where they number at most a CU's one each, or, with
//  kTallRows or more rows an expert, where 128 x 256 tiles would take at most one
//  and a half rounds: against the persistent kernel at E = 8, N = K = 2048, mean
//  72: 15.5 / 20.6, 200: 17.2 / 22.9, 500: 34.9 / 40.2; E = 64, N x K = 512 x
//  2560, mean 24: 24.1 / 31.9; E = 4, N x K = 5120 x 2048, mean 500: 34.2 / 43.0.
//  Elsewhere the persistent kernel: against 128 x 128 tiles at E = 40, N x K =
//  5120 x 1408, mean 16: 59.1 / 67.3, 48: 70.3 / 80.1, 80: 77.0 / 89.9; E = 32,
//  N x K = 2048 x 5120, mean 24: 63.9 / 61.8, 80: 104.3 / 111.6.
constexpr uint32_t kTileMinRows = 14, kFewTilesMaxRows = 64, kTallRows = 192;

int group_auto(uint32_t R, uint32_t E, uint32_t N, uint32_t cus) {
  const uint32_t groups = R < E ? R : E;
  if (groups == 0) return kGroupStream;
  const uint32_t mean = R / groups;
  const bool few = (uint64_t)groups * (N / 128) < cus;
  if (mean < (few ? kFewTilesMaxRows : kTileMinRows)) return kGroupStream;
  // row tiles: half a tile an expert more than its rows fill
  const uint64_t rt = std::max<uint64_t>(groups, ((uint64_t)R + 64ull * groups) / 128);
  if (rt * (N / 128) <= cus || (mean >= kTallRows && 2 * rt * ((N + 255) / 256) <= 3ull * cus)) return kGroupTiled;
  return kGroupPp;
}

// The streaming form.  Rows a tile: 16 up to a mean of kStreamFewRows rows an
// expert, else 32.  A stage is 16 KB of weights: 128 columns x 1 K block where
// every worker has at least kWideGranules granules, 64 x 2 from kMidGranules on,
// else 32 x 4 (narrower stages would leave waves without columns).  us at
// 64 x 2 / 128 x 1 / 32 x 4: E = 32, N x K = 2048 x 5120 (16 granules a worker),
// mean 8: 60.7 / 54.3 / -; E = 8 (4 granules), mean 2: 14.8 / 14.9 / 15.3;
// E = 4 (2 granules), mean 2: 11.4 / 11.4 / 8.7; one expert, N x K = 5120 x
// 17408, 16 rows: 32.7 / 53.3 / 23.5.
constexpr uint32_t kStreamFewRows = 4, kWideGranules = 6, kMidGranules = 3;

template <bool F16>
hipError_t launch_stream_any(const uint8_t* a, const float* as, const GroupWeights& gw, uint32_t sets,
                             const Groups& g, uint32_t N, uint32_t K, uint32_t cus, hipStream_t s) {
  const uint64_t per_worker = (uint64_t)(g.R < g.E ? g.R : g.E) * sets * (N / 16) / cus;
  if ((uint64_t)g.R <= (uint64_t)kStreamFewRows * g.E)
    return per_worker >= kMidGranules ? launch_stream<1, 1, 4, 2, F16>(a, as, gw, sets, g, N, K, cus, s)
                                      : launch_stream<1, 1, 2, 4, F16>(a, as, gw, sets, g, N, K, cus, s);
  if (per_worker >= kWideGranules) return launch_stream<2, 1, 8, 1, F16>(a, as, gw, sets, g, N, K, cus, s);
  return per_worker >= kMidGranules ? launch_stream<2, 1, 4, 2, F16>(a, as, gw, sets, g, N, K, cus, s)
                                    : launch_stream<2, 1, 2, 4, F16>(a, as, gw, sets, g, N, K, cus, s);
}

hipError_t launch_any(const uint8_t* a, const float* as, const GroupWeights& gw, uint32_t sets,
                      const Groups& g, uint32_t N, uint32_t K, uint32_t cus, int kernel, hipStream_t s) {
  // mostly one row tile an expert: its weights are read once
  const bool once = g.R < (uint64_t)kReadOnceRows * g.E;
  switch (kernel) {
    // two sets: gate and up, in f16.  One product's result is only rounded to bf16
    // (2^-9), which hides the FP8 sums' 1.4e-5: 3.7e-4 of its norm from that rounding
    // of the 64-bit value.
    case kGroupStream:
      return sets == 2 ? launch_stream_any<true>(a, as, gw, sets, g, N, K, cus, s)
                       : launch_stream_any<false>(a, as, gw, sets, g, N, K, cus, s);
    case kGroupPp:
      if (sets == 1 && g.E <= kPersistMaxExperts && K >= kPersistMinBlocks * kGroup)
        return once ? launch_group_persist<kStreamOnce>(a, as, gw, g, N, K, cus, s)
                    : launch_group_persist<0>(a, as, gw, g, N, K, cus, s);
      break;
    default: break;
  }
  return once ? launch_group_128<kStreamOnce>(a, as, gw, sets, g, N, K, s)
              : launch_group_128<0>(a, as, gw, sets, g, N, K, s);
}

}  // namespace

int group_gemm_auto(uint32_t R, uint32_t E, uint32_t N, uint32_t cus) { return group_auto(R, E, N, cus); }

hipError_t launch_gemm_grouped(const uint8_t* a, const float* a_s_km, const uint8_t* w,
                               const float* w_s, uint16_t* out, const int32_t* offsets,
                               const int32_t* order, uint32_t per_row, uint32_t a_rows, uint32_t R,
                               uint32_t E, uint32_t N, uint32_t K, uint32_t cus, int kernel,
                               hipStream_t s) {
  return launch_any(a, a_s_km, GroupWeights{{w, w}, {w_s, w_s}, {out, out}}, 1,
                    Groups{offsets, order, E, R, per_row, a_rows}, N, K, cus, kernel, s);
}

hipError_t launch_group_gate_and_up(const uint8_t* x, const float* x_s_km, const uint8_t* w_gate,
                                    const float* ws_gate, const uint8_t* w_up, const float* ws_up,
                                    uint16_t* gate, uint16_t* up, const int32_t* offsets,
                                    const int32_t* order, uint32_t per_row, uint32_t a_rows, uint32_t R,
                                    uint32_t E, uint32_t H, uint32_t I, uint32_t cus, int kernel,
                                    hipStream_t s) {
  return launch_any(x, x_s_km, GroupWeights{{w_gate, w_up}, {ws_gate, ws_up}, {gate, up}}, 2,
                    Groups{offsets, order, E, R, per_row, a_rows}, I, H, cus, kernel, s);
}

namespace {
hipError_t launch_gate_up(const uint8_t* x, const float* x_s_km, const GroupWeights& gw, const FfnArgs& f,
                          const Groups& g, uint32_t H, uint32_t I, hipStream_t s) {
  using C = PpCfg<3, false, true>;
  const hipError_t e = allow_lds<&group_gate_up_kernel, C::LDS_BYTES>();
  if (e != hipSuccess) return e;
  const uint32_t tiles_n = I / kGroup;
  group_gate_up_kernel<<<dim3(max_row_tiles(g.R, g.E, C::BM) * tiles_n), dim3(C::NT), C::LDS_BYTES, s>>>(
      x, x_s_km, gw, g, f.hq, f.hs, I, H, m_pad16(g.a_rows), f.Mp_h, tiles_n);
  return hipGetLastError();
}

template <int WAUX>
hipError_t launch_persist_ffn(const uint8_t* x, const float* x_s_km, const GroupWeights& gw, const FfnArgs& f,
                              const Groups& g, uint32_t H, uint32_t I, uint32_t cus, hipStream_t s) {
  const hipError_t e = allow_lds<&group_persist_ffn_kernel<WAUX>, PersistCfg::LDS>();
  if (e != hipSuccess) return e;
  const uint32_t tiles_n = I / kGroup;
  const uint64_t most = (uint64_t)max_row_tiles(g.R, g.E, 128) * tiles_n;
  group_persist_ffn_kernel<WAUX><<<dim3((uint32_t)(most < cus ? most : cus)), dim3(512), PersistCfg::LDS, s>>>(
      x, x_s_km, gw.w[0], gw.ws[0], f, g, I, H, m_pad16(g.a_rows), tiles_n);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_group_ffn_gate_up(const uint8_t* x, const float* x_s_km, const uint8_t* w_gate,
                                    const float* ws_gate, const uint8_t* w_up, const float* ws_up,
                                    uint8_t* hq, float* hs_km, const int32_t* offsets,
                                    const int32_t* order, uint32_t per_row, uint32_t a_rows, uint32_t R,
                                    uint32_t E, uint32_t H, uint32_t I, uint32_t cus, hipStream_t s) {
  const GroupWeights gw{{w_gate, w_up}, {ws_gate, ws_up}, {nullptr, nullptr}};
  const Groups g{offsets, order, E, R, per_row, a_rows};
  const FfnArgs f{w_up, ws_up, hq, hs_km, m_pad16(R)};
  if (E > kPersistMaxExperts || H < kPersistMinBlocks * kGroup) return launch_gate_up(x, x_s_km, gw, f, g, H, I, s);
  return R < (uint64_t)kReadOnceRows * E ? launch_persist_ffn<kStreamOnce>(x, x_s_km, gw, f, g, H, I, cus, s)
                                         : launch_persist_ffn<0>(x, x_s_km, gw, f, g, H, I, cus, s);
}

}  // namespace fp8q
