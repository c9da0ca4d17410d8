// Products grouped by expert on gfx950 (block-scaled FP8):
//   out[p, n] = bf16( sum_kb a_s[kb][r] * w_s[e][n/128][kb] * P(r, e, n, kb) ),
//   r = order[p] / per_row (or p), e: offsets[e] <= p < offsets[e + 1],
// with P the 128-deep e4m3 dot products of the dense GEMM (gemm.hip).
#include <atomic>

#include "gemm_pp.h"
#include "group_tiles.h"

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
// reading each active expert's weights once from HBM.  A wave owns 16 output
// columns (16 weight rows) and streams its K range through an LDS ring of its
// own with direct loads, so there is no workgroup barrier in the loop; each
// load instruction covers two weight rows x 512 contiguous bytes (whole cache
// lines).  Ring buffer: 16 rows x 4 K blocks, 16-byte chunk c of a row at
// position c ^ swz(row) within its K block, as in the tiled kernel.  The
// activation fragments (16 * TM rows, most of them of other tokens: rows past
// the group load as zeros, without a memory access) come from L2 into
// registers one chunk ahead.
//
// KS waves share 16 columns, each a contiguous part of K; their partial tiles
// are added in K order through LDS at the end.
// ------------------------------------------------------------------------
constexpr int kStreamBlocks = 4;                             // K blocks per ring buffer
constexpr int kStreamBuf = 16 * kStreamBlocks * 128;         // 8 KB
// past any operand's bound (ceil16(rows) * K < 2^32, so at most 0xFFFFF800), also 16 bytes on
constexpr uint32_t kOutOfRange = 0xFFFFFF00u;

template <int TM, int WAVES, int KS>
__global__ __launch_bounds__(64 * WAVES) void group_stream_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ As, GroupWeights gw, Groups g,
    uint32_t N, uint32_t K, uint32_t Mp, uint32_t tiles_n) {
  constexpr int CW = WAVES / KS, CB = kStreamBlocks;  // column tiles a workgroup, K blocks a chunk
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  GroupTile t;
  if (!group_tile<16 * TM>(g, tiles_n, blockIdx.x, lane, t)) return;
  const uint32_t l16 = lane & 15, q = lane >> 4, G = K / kGroup;
  const uint32_t cw = wave % CW, ks = wave / CW;
  const uint32_t n0 = (t.tn * CW + cw) * 16;
  const uint32_t kbeg = ks * G / KS, kend = (ks + 1) * G / KS;
  const uint32_t which = blockIdx.y;
  const uint8_t* W = gw.w[which] + ((uint64_t)t.expert * N + n0) * K;
  const float* Ws = gw.ws[which] + ((uint64_t)t.expert * (N / kGroup) + n0 / kGroup) * G;
  const GroupRows rows{g.a_rows, t.end, g.order, g.per_row};

  const __amdgpu_buffer_rsrc_t rA = make_rsrc(A, g.a_rows * K);
  const __amdgpu_buffer_rsrc_t rW = make_rsrc(W, 16 * K);
  uint32_t a_off[TM], s_idx[TM];
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const uint32_t m = t.m0 + 16 * tm + l16;
    const uint32_t r = rows.src(min(m, t.end - 1));
    a_off[tm] = m < t.end ? r * K + 32 * q : kOutOfRange;
    s_idx[tm] = r;
  }
  // source of this lane's 16 bytes in load j of a chunk: weight row 2j + lane/32,
  // chunk position lane % 32
  const uint32_t pos = lane & 31, blk = pos >> 3;
  const uint32_t ring = lds_addr(smem) + wave * 2 * kStreamBuf;
  uint32_t w_off[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t row = 2 * j + (lane >> 5);
    w_off[j] = row * K + blk * kGroup + ((pos & 7) ^ swz(row)) * 16;
  }
  auto issue_w = [&](uint32_t kb, uint32_t buf) __attribute__((always_inline)) {
    const uint32_t out = kb + blk < kend ? 0 : kOutOfRange;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      dma16_at(rW, w_off[j] | out, kb * kGroup, ring + buf * kStreamBuf + j * 1024);
  };
  struct Frag {
    v8i a[CB][TM];
    float as[CB][TM], ws;  // ws: lane b holds the weight scale of block b (b < CB)
  };
  auto load_a = [&](Frag& f, uint32_t kb) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < CB; ++b) {
      const uint32_t k = min(kb + b, kend - 1);  // past the range: the weights are zeros
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        f.a[b][tm] = join(__builtin_amdgcn_raw_buffer_load_b128(rA, a_off[tm], k * kGroup, 0),
                          __builtin_amdgcn_raw_buffer_load_b128(rA, a_off[tm] + 16, k * kGroup, 0));
        f.as[b][tm] = As[(uint64_t)k * Mp + s_idx[tm]];
      }
    }
    f.ws = Ws[min(kb + (lane & (CB - 1)), kend - 1)];
  };
  v4f acc[TM];
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) acc[tm] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const uint32_t c0 = 2 * q;
  const uint32_t lo0 = l16 * (CB * 128) + ((c0 ^ swz(l16)) * 16);
  const uint32_t lo1 = l16 * (CB * 128) + (((c0 + 1) ^ swz(l16)) * 16);
  const uint8_t* my = smem + wave * 2 * kStreamBuf;
  auto consume = [&](const Frag& f, uint32_t buf) __attribute__((always_inline)) {
    const uint8_t* s = my + buf * kStreamBuf;
    v8i w[CB];
#pragma unroll
    for (int b = 0; b < CB; ++b) {
      w[b] = join(*reinterpret_cast<const u32x4*>(s + lo0 + b * 128),
                  *reinterpret_cast<const u32x4*>(s + lo1 + b * 128));
    }
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      v4f p[CB];
#pragma unroll
      for (int b = 0; b < CB; ++b) p[b] = mfma_e4m3_128(w[b], f.a[b][tm]);
#pragma unroll
      for (int b = 0; b < CB; ++b)
        acc[tm] += p[b] * (f.as[b][tm] * __uint_as_float((uint32_t)__builtin_amdgcn_readlane(
                                             (int)__float_as_uint(f.ws), b)));
    }
  };
  if (kbeg < kend) {
    // Loads are issued chunk by chunk, weights then activations, in this
    // order (the fences): at most the next chunk's 8 + 12 * TM + 1 may be
    // outstanding when a chunk is consumed.
    constexpr int AHEAD = 8 + CB * 3 * TM + 1;
    Frag f0, f1;
    auto issue = [&](Frag& f, uint32_t kb, uint32_t buf) __attribute__((always_inline)) {
      sched_fence();
      issue_w(kb, buf);  // past the range: zeros, no memory access
      sched_fence();
      load_a(f, min(kb, kend - 1));
      sched_fence();
    };
    issue(f0, kbeg, 0);
    issue(f1, kbeg + CB, 1);
    for (uint32_t kb = kbeg; kb < kend; kb += 2 * CB) {
      wait_vmcnt<AHEAD>();
      consume(f0, 0);
      wait_lgkm0();
      issue(f0, kb + 2 * CB, 0);
      wait_vmcnt<AHEAD>();
      consume(f1, 1);
      wait_lgkm0();
      issue(f1, kb + 3 * CB, 1);
    }
    wait_vmcnt<0>();  // no direct load may still be writing LDS
  }
  if constexpr (KS > 1) {
    wg_barrier();
    v4f* red = reinterpret_cast<v4f*>(smem);
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) red[(wave * TM + tm) * 64 + lane] = acc[tm];
    __syncthreads();
    if (ks != 0) return;
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)
#pragma unroll
      for (int k = 1; k < KS; ++k) acc[tm] += red[((k * CW + cw) * TM + tm) * 64 + lane];
  }
  uint16_t* out = gw.out[which];
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const uint32_t m = t.m0 + 16 * tm + l16;
    if (m < t.end) *reinterpret_cast<uint2*>(out + (uint64_t)m * N + n0 + 4 * q) = pack_bf16x4(acc[tm]);
  }
}

template <int TM, int WAVES, int KS>
hipError_t launch_stream(const uint8_t* a, const float* as, const GroupWeights& gw, uint32_t sets,
                         const Groups& g, uint32_t N, uint32_t K, hipStream_t s) {
  constexpr uint32_t LDS = WAVES * 2 * kStreamBuf;
  static_assert(LDS <= 64 * 1024 && WAVES * TM * 1024 <= (int)LDS, "ring, partial tiles");
  const uint32_t tiles_n = N / (16 * (WAVES / KS));
  const uint32_t grid = max_row_tiles(g.R, g.E, 16 * TM) * tiles_n;
  group_stream_kernel<TM, WAVES, KS><<<dim3(grid, sets), dim3(64 * WAVES), LDS, s>>>(
      a, as, gw, g, N, K, m_pad16(g.a_rows), tiles_n);
  return hipGetLastError();
}

// ------------------------------------------------------------------------
// The dense GEMM's tiled and ping-pong kernels over the experts' rows.
// ------------------------------------------------------------------------
template <int BM, int BN, int WGM, int WGN, int STAGES>
__global__ __launch_bounds__(64 * WGM * WGN) void group_tiled_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ As, GroupWeights gw, Groups g,
    uint32_t N, uint32_t K, uint32_t Mp, uint32_t tiles_n) {
  GroupTile t;
  if (!group_tile<BM>(g, tiles_n, blockIdx.x, threadIdx.x & 63, t)) return;
  const uint32_t which = blockIdx.y;
  gemm_tiled_body<BM, BN, WGM, WGN, STAGES, false, false>(
      A, As, gw.w[which] + (uint64_t)t.expert * N * K,
      gw.ws[which] + (uint64_t)t.expert * (N / kGroup) * (K / kGroup), gw.out[which], t.m0, t.tn * BN,
      N, K, Mp, 0, 1, nullptr, GroupRows{g.a_rows, t.end, g.order, g.per_row}, NoEpilogue{});
}

__global__ __launch_bounds__(512) void group_pp_kernel(const uint8_t* __restrict__ A,
                                                       const float* __restrict__ As, GroupWeights gw,
                                                       Groups g, uint32_t N, uint32_t K, uint32_t Mp,
                                                       uint32_t tiles_n) {
  using C = PpCfg<3, false, false>;
  GroupTile t;
  if (!group_tile<C::BM>(g, tiles_n, blockIdx.x, threadIdx.x & 63, t)) return;
  const uint32_t which = blockIdx.y;
  gemm_pp_body<3, false, false>(A, As, gw.w[which] + (uint64_t)t.expert * N * K,
                                gw.ws[which] + (uint64_t)t.expert * (N / kGroup) * (K / kGroup),
                                gw.out[which], t.m0, t.tn * C::BN, N, K, Mp,
                                FfnArgs{nullptr, nullptr, nullptr, nullptr, 0},
                                GroupRows{g.a_rows, t.end, g.order, g.per_row}, NoEpilogue{});
}

// Fused gate/up of the experts' FFN: the ping-pong kernel's FFN mode, 128
// sorted rows by 128 intermediate columns, writing the quantized intermediate.
__global__ __launch_bounds__(512) void group_gate_up_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ As, GroupWeights gw, Groups g,
    uint8_t* __restrict__ hq, float* __restrict__ hs, uint32_t I, uint32_t H, uint32_t Mp,
    uint32_t Mp_h, uint32_t tiles_n) {
  using C = PpCfg<3, false, true>;
  GroupTile t;
  if (!group_tile<C::BM>(g, tiles_n, blockIdx.x, threadIdx.x & 63, t)) return;
  const uint64_t wo = (uint64_t)t.expert * I * H, so = (uint64_t)t.expert * (I / kGroup) * (H / kGroup);
  gemm_pp_body<3, false, true>(A, As, gw.w[0] + wo, gw.ws[0] + so, nullptr, t.m0, t.tn * kGroup, I, H,
                               Mp, FfnArgs{gw.w[1] + wo, gw.ws[1] + so, hq, hs, Mp_h},
                               GroupRows{g.a_rows, t.end, g.order, g.per_row}, NoEpilogue{});
}

template <class F>
hipError_t allow_lds(std::atomic<bool>& done, F* kernel, int bytes) {
  if (done.load(std::memory_order_acquire)) return hipSuccess;  // idempotent: racing threads repeat it
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.store(true, std::memory_order_release);
  return e;
}

hipError_t launch_group_128(const uint8_t* a, const float* as, const GroupWeights& gw, uint32_t sets,
                            const Groups& g, uint32_t N, uint32_t K, hipStream_t s) {
  using C = TileCfg<128, 128, 2, 2, 2, false>;
  static std::atomic<bool> done{false};
  const hipError_t e = allow_lds(done, &group_tiled_kernel<128, 128, 2, 2, 2>, C::LDS_BYTES);
  if (e != hipSuccess) return e;
  const uint32_t tiles_n = N / 128;
  group_tiled_kernel<128, 128, 2, 2, 2><<<dim3(max_row_tiles(g.R, g.E, 128) * tiles_n, sets), dim3(C::NT),
                                          C::LDS_BYTES, s>>>(a, as, gw, g, N, K, m_pad16(g.a_rows), tiles_n);
  return hipGetLastError();
}

hipError_t launch_group_pp(const uint8_t* a, const float* as, const GroupWeights& gw, uint32_t sets,
                           const Groups& g, uint32_t N, uint32_t K, hipStream_t s) {
  using C = PpCfg<3, false, false>;
  static std::atomic<bool> done{false};
  const hipError_t e = allow_lds(done, &group_pp_kernel, C::LDS_BYTES);
  if (e != hipSuccess) return e;
  const uint32_t tiles_n = N / C::BN;
  group_pp_kernel<<<dim3(max_row_tiles(g.R, g.E, C::BM) * tiles_n, sets), dim3(C::NT), C::LDS_BYTES, s>>>(
      a, as, gw, g, N, K, m_pad16(g.a_rows), tiles_n);
  return hipGetLastError();
}

// Kernel ids of the grouped product
constexpr int kGroupStream = 1, kGroupTiled = 2, kGroupPp = 3;

int group_auto(uint32_t R, uint32_t E) {
  const uint32_t mean = R / (R < E ? R : E);  // rows per expert at least
  return mean <= 16 ? kGroupStream : mean < 192 ? kGroupTiled : kGroupPp;
}

hipError_t launch_any(const uint8_t* a, const float* as, const GroupWeights& gw, uint32_t sets,
                      const Groups& g, uint32_t N, uint32_t K, uint32_t cus, int kernel, hipStream_t s) {
  switch (kernel) {
    case kGroupStream: {
      // K split until the grid holds about two workgroups per CU
      const uint64_t wgs = (uint64_t)(g.R < g.E ? g.R : g.E) * sets * (N / 64);
      if (wgs >= 2 * cus) return launch_stream<1, 4, 1>(a, as, gw, sets, g, N, K, s);
      if (2 * wgs >= 2 * cus) return launch_stream<1, 4, 2>(a, as, gw, sets, g, N, K, s);
      return launch_stream<1, 4, 4>(a, as, gw, sets, g, N, K, s);
    }
    case kGroupTiled: return launch_group_128(a, as, gw, sets, g, N, K, s);
    default: return launch_group_pp(a, as, gw, sets, g, N, K, s);
  }
}

Groups make_groups(const int32_t* offsets, const int32_t* order, uint32_t E, uint32_t R,
                   uint32_t per_row, uint32_t a_rows) {
  return Groups{offsets, order, E, R, per_row, a_rows};
}

}  // namespace

int group_gemm_auto(uint32_t R, uint32_t E) { return group_auto(R, E); }

hipError_t launch_gemm_grouped(const uint8_t* a, const float* a_s_km, const uint8_t* w,
                               const float* w_s, uint16_t* out, const int32_t* offsets,
                               const int32_t* order, uint32_t per_row, uint32_t a_rows, uint32_t R,
                               uint32_t E, uint32_t N, uint32_t K, uint32_t cus, int kernel,
                               hipStream_t s) {
  return launch_any(a, a_s_km, GroupWeights{{w, w}, {w_s, w_s}, {out, out}}, 1,
                    make_groups(offsets, order, E, R, per_row, a_rows), N, K, cus, kernel, s);
}

hipError_t launch_group_gate_and_up(const uint8_t* x, const float* x_s_km, const uint8_t* w_gate,
                                    const float* ws_gate, const uint8_t* w_up, const float* ws_up,
                                    uint16_t* gate, uint16_t* up, const int32_t* offsets,
                                    const int32_t* order, uint32_t per_row, uint32_t a_rows, uint32_t R,
                                    uint32_t E, uint32_t H, uint32_t I, uint32_t cus, int kernel,
                                    hipStream_t s) {
  return launch_any(x, x_s_km, GroupWeights{{w_gate, w_up}, {ws_gate, ws_up}, {gate, up}}, 2,
                    make_groups(offsets, order, E, R, per_row, a_rows), I, H, cus, kernel, s);
}

hipError_t launch_group_ffn_gate_up(const uint8_t* x, const float* x_s_km, const uint8_t* w_gate,
                                    const float* ws_gate, const uint8_t* w_up, const float* ws_up,
                                    uint8_t* hq, float* hs_km, const int32_t* offsets,
                                    const int32_t* order, uint32_t per_row, uint32_t a_rows, uint32_t R,
                                    uint32_t E, uint32_t H, uint32_t I, hipStream_t s) {
  using C = PpCfg<3, false, true>;
  static std::atomic<bool> done{false};
  const hipError_t e = allow_lds(done, &group_gate_up_kernel, C::LDS_BYTES);
  if (e != hipSuccess) return e;
  const uint32_t tiles_n = I / kGroup;
  group_gate_up_kernel<<<dim3(max_row_tiles(R, E, C::BM) * tiles_n), dim3(C::NT), C::LDS_BYTES, s>>>(
      x, x_s_km, GroupWeights{{w_gate, w_up}, {ws_gate, ws_up}, {nullptr, nullptr}},
      make_groups(offsets, order, E, R, per_row, a_rows), hq, hs_km, I, H, m_pad16(a_rows), m_pad16(R),
      tiles_n);
  return hipGetLastError();
}

}  // namespace fp8q
