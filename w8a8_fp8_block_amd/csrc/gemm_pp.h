// The ping-pong block-scaled FP8 GEMM: configuration, FFN epilogue and the
// kernel body, shared by the dense kernels (gemm.hip), the expert-grouped ones
// (grouped.hip) and the projection with per-request adapters (lora.hip).
#pragma once

#include "gemm_tile.h"
#include "quant_common.h"

namespace fp8q {
namespace {

// ------------------------------------------------------------------------
// Ping-pong kernel: 256x128 workgroup tile, 8 waves of 64x64 in two groups.
// Group 0 (waves 0-3, tile rows 0-127) and group 1 (waves 4-7, rows
// 128-255) put one wave on each SIMD and take turns: while one group runs
// the MFMAs and promotions of a K block from registers, the other reads its
// fragments of the block from LDS, so each SIMD's matrix pipe is fed by one
// wave at a time instead of two waves that leave every barrier together and
// compete.  Per K block kb:
//   phase A: group 0 computes block kb; group 1 reads block kb
//   phase B: group 1 computes block kb; group 0 reads block kb+1
// with a workgroup barrier after each phase.  A wave holds one fragment set
// (loaded in its read phase, consumed in its compute phase).
//
// Direct loads: a stage is 48 1-KB operand chunks (chunk c at LDS offset
// c*1024: activation rows 8c..8c+7 for c < 32, weight rows 8(c-32).. after)
// plus every wave's scales.  Each wave issues 8 loads per block at the end
// of its read phase (group 0: 8 operand chunks; group 1: 4 chunks and the
// scales of two waves), so the texture unit gets 32 or 16 KB per phase and
// the compute phases hold nothing but MFMAs and promotions.  Stage s
// (block min(s, G-1): stages past the last block reload it, in bounds and
// never read) goes to slot s % STAGES.  Before the phase-A barrier of block
// kb each wave waits for its own part of stage kb+1.
//
// FFN mode (the dense FFN's fused gate/up projection): the workgroup tile is
// 128 token rows by 256 weight rows, the 128 gate rows n0.. and the 128 up
// rows n0.. of one intermediate column block; group 0 computes gate and group
// 1 up, wave for wave on the same 64x64 output positions, and the epilogue
// forms h = bf16(silu(bf16 gate) * bf16 up), quantizes it per (token,
// 128-group) and writes the codes and the K-major scales (see
// ffn_epilogue).  The main loop is the same code with the weight chunks
// read from two sources.
// ------------------------------------------------------------------------
template <int STAGES, bool ROW = false, bool FFN = false>
struct PpCfg {
  static constexpr int BM = FFN ? 128 : 256, BN = FFN ? 256 : 128, NW = 8, NT = 512;
  static constexpr int WM = 64, WN = 64, TM = 4, TN = 4, NP = 16;
  static constexpr int A_BYTES = BM * 128, W_BYTES = BN * 128;
  static constexpr int SCW_BYTES = 512;  // per wave: 64 activation scales + 64 weight-scale copies
  static constexpr int STAGE_BYTES = A_BYTES + W_BYTES + NW * SCW_BYTES;
  static constexpr int LDS_BYTES = STAGES * STAGE_BYTES;
  static constexpr int CHUNKS = (A_BYTES + W_BYTES) / 1024;  // 48
  // loads per wave and stage: group 0 eight operand chunks; group 1 four
  // operand chunks and the scales of itself and of its group-0 partner
  static constexpr int CH0 = 8, CH1 = 4;
  static constexpr int LW0 = CH0, LW1 = CH1 + 2 * (ROW ? 1 : 2);
  static_assert(4 * (CH0 + CH1) == CHUNKS && 2 * LW1 < 64, "chunk split, vmcnt range");
  static_assert(LDS_BYTES <= 160 * 1024 && STAGES == 3, "config");
  static_assert(kPromoteDist >= 1 && kPromoteDist <= 3 && kPromoteDist <= TN && NP % 4 == 0,
                "pending promotions lie in the last row; four result registers");
};

// Second weight operand and outputs of the FFN mode: W/Ws are the gate
// weights and their block scales, these the up weights and scales, the
// intermediate's codes [M,N] and its K-major scales [N/128, Mp_h].
struct FfnArgs {
  const uint8_t* w_up;
  const float* ws_up;
  uint8_t* hq;
  float* hs;
  uint32_t Mp_h;  // row stride of hs
};

// FFN-mode epilogue.  Gate wave gw (group 0) and up wave gw (group 1, wave gw +
// 4) hold the same 64x64 output positions in the same registers; they split the
// rows: the gate wave finishes rows tm = 0, 1 of its band, the up wave rows tm =
// 2, 3.
//   1. ffn_park: each wave rounds its accumulators to bf16 (the projections'
//      output format) and parks the half its partner finishes in LDS (32 KB);
//   2. ffn_h: each wave forms h = bf16(silu(g) * u) for its rows (silu_mul_f32,
//      the same code as the standalone intermediate kernel) and the maximum |h|
//      of each row over its 64 columns (integer max of bf16 magnitudes: within a
//      lane, then across the 4 lanes of a row), left in LDS (512 bytes);
//   3. ffn_codes: the two waves of a group covering columns 0-63 and 64-127 of
//      the 128-column group combine their row maxima; scale = amax/448 and the
//      codes of h / scale follow the activation quantizer's exact steps
//      (quotients, encode4).  Codes of rows < M are stored; the wave on columns
//      0-63 stores the K-major scales of its rows < M and zeros for pad rows M
//      .. pad_end-1.
// A workgroup barrier between the steps, each after the LDS writes before it
// have completed (s_barrier alone does not wait for them).
constexpr uint32_t kFfnPark = 32 * 1024, kFfnMax = 8 * 2 * 16 * 2;

template <int TM, int TN>
__device__ __forceinline__ void ffn_park(const v4f (&acc)[TM][TN], uint8_t* smem, uint32_t wave, uint32_t lane) {
  static_assert(TM == 4 && TN == 4, "64x64 wave tile");
  uint32_t* park = reinterpret_cast<uint32_t*>(smem);  // [8][4][64][4] u32
  const bool up = wave >= 4;
  // the tiles of rows tm = 0, 1 (up waves) or 2, 3 (gate waves), two 16x16
  // tiles per 16-byte slot
#pragma unroll
  for (int t2 = 0; t2 < 4; ++t2) {
    const int t = 2 * t2;  // tile index within the half
    const uint2 a = up ? pack_bf16x4(acc[t / TN][t % TN]) : pack_bf16x4(acc[2 + t / TN][t % TN]);
    const uint2 b = up ? pack_bf16x4(acc[(t + 1) / TN][(t + 1) % TN])
                       : pack_bf16x4(acc[2 + (t + 1) / TN][(t + 1) % TN]);
    *reinterpret_cast<uint4*>(park + ((wave * 4 + t2) * 64 + lane) * 4) = make_uint4(a.x, a.y, b.x, b.y);
  }
}

// hb: h as packed bf16 pairs, rows i = 0, 1 of this wave's half
template <int TM, int TN>
__device__ __forceinline__ void ffn_h(const v4f (&acc)[TM][TN], const uint8_t* smem, uint16_t* rmax, uint32_t wave,
                                      uint32_t lane, uint32_t (&hb)[2][TN][2], uint32_t (&amax)[2]) {
  const uint32_t* park = reinterpret_cast<const uint32_t*>(smem);
  const uint32_t l16 = lane & 15, q4 = lane >> 4, partner = wave ^ 4;
  const bool up = wave >= 4;
#pragma unroll
  for (int t2 = 0; t2 < 4; ++t2) {
    const uint4 pp = *reinterpret_cast<const uint4*>(park + ((partner * 4 + t2) * 64 + lane) * 4);
    const uint32_t pw[4] = {pp.x, pp.y, pp.z, pp.w};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = 2 * t2 + h, i = t / TN, tn = t % TN;
      const uint2 own = up ? pack_bf16x4(acc[2 + i][tn]) : pack_bf16x4(acc[i][tn]);
      const uint32_t ow[2] = {own.x, own.y};
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const uint32_t g2 = up ? pw[2 * h + d] : ow[d], u2 = up ? ow[d] : pw[2 * h + d];
        const float lo = silu_mul_f32(__uint_as_float(g2 << 16), __uint_as_float(u2 << 16));
        const float hi = silu_mul_f32(__uint_as_float(g2 & 0xFFFF0000u), __uint_as_float(u2 & 0xFFFF0000u));
        hb[i][tn][d] = bf16x2_rne(lo, hi);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t mx = 0;
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) {
      const uint32_t a = hb[i][tn][0] & 0x7FFF7FFFu, b = hb[i][tn][1] & 0x7FFF7FFFu;
      mx = max(mx, max(max(a & 0xFFFFu, a >> 16), max(b & 0xFFFFu, b >> 16)));
    }
    mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16));
    mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32));
    amax[i] = mx;
    if (q4 == 0) rmax[(wave * 2 + i) * 16 + l16] = (uint16_t)mx;
  }
}

template <int TN>
__device__ __forceinline__ void ffn_codes(const uint32_t (&hb)[2][TN][2], const uint32_t (&amax)[2],
                                          const uint16_t* rmax, const FfnArgs& ffn, uint32_t wave, uint32_t lane,
                                          uint32_t mrow0, uint32_t ncol0, uint32_t nb, uint32_t M, uint32_t N,
                                          uint32_t pad_end) {
  const uint32_t l16 = lane & 15, q4 = lane >> 4;
  const uint32_t mate = wave ^ 1;  // the other 64 columns of the 128-column group
  const bool up = wave >= 4;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = max(amax[i], (uint32_t)rmax[(mate * 2 + i) * 16 + l16]);
    const float sc = group_scale(a);
    float x[16], q[16];
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) {
      x[4 * tn + 0] = __uint_as_float(hb[i][tn][0] << 16);
      x[4 * tn + 1] = __uint_as_float(hb[i][tn][0] & 0xFFFF0000u);
      x[4 * tn + 2] = __uint_as_float(hb[i][tn][1] << 16);
      x[4 * tn + 3] = __uint_as_float(hb[i][tn][1] & 0xFFFF0000u);
    }
    quotients<16>(x, sc, q);
    const uint32_t m = mrow0 + ((up ? 2 : 0) + i) * 16 + l16;
    if (m < M) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
        *reinterpret_cast<uint32_t*>(ffn.hq + (uint64_t)m * N + ncol0 + tn * 16 + 4 * q4) =
            encode4(q + 4 * tn);
    }
    if ((wave & 1) == 0 && q4 == 0 && m < pad_end) ffn.hs[(uint64_t)nb * ffn.Mp_h + m] = (m < M) ? sc : 0.0f;
  }
}

// The whole of it after the main loop (all direct loads of this wave complete):
// every wave passes the same three workgroup barriers.
template <int TM, int TN>
__device__ __forceinline__ void ffn_epilogue(const v4f (&acc)[TM][TN], uint8_t* smem,
                                             const FfnArgs& ffn, uint32_t wave, uint32_t lane,
                                             uint32_t mrow0, uint32_t ncol0, uint32_t nb,
                                             uint32_t M, uint32_t N, uint32_t pad_end) {
  uint16_t* rmax = reinterpret_cast<uint16_t*>(smem + kFfnPark);
  auto lds_barrier = [] {
    wait_lgkm0();
    wg_barrier();
  };
  lds_barrier();  // every wave is done with the operand ring
  ffn_park<TM, TN>(acc, smem, wave, lane);
  lds_barrier();
  uint32_t hb[2][TN][2], amax[2];
  ffn_h<TM, TN>(acc, smem, rmax, wave, lane, hb, amax);
  lds_barrier();
  ffn_codes<TN>(hb, amax, rmax, ffn, wave, lane, mrow0, ncol0, nb, M, N, pad_end);
}

template <int STAGES, bool ROW, bool FFN, class Rows, class Epi>
__device__ __forceinline__ void gemm_pp_body(
    const uint8_t* __restrict__ A, const float* __restrict__ As, const uint8_t* __restrict__ W,
    const float* __restrict__ Ws, uint16_t* __restrict__ out, uint32_t m0, uint32_t n0, uint32_t N,
    uint32_t K, uint32_t Mp, const FfnArgs& ffn, const Rows& rows, const Epi& epi) {
  using C = PpCfg<STAGES, ROW, FFN>;
  constexpr int TM = C::TM, TN = C::TN, NP = C::NP;
  constexpr int CH0 = C::CH0, CH1 = C::CH1, LW0 = C::LW0, LW1 = C::LW1;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];

  const uint32_t tid = threadIdx.x, lane = tid & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t grp = wave >> 2, gw = wave & 3;
  const uint32_t wm = FFN ? gw >> 1 : 2 * grp + (gw >> 1);
  const uint32_t wn = FFN ? 2 * grp + (gw & 1) : gw & 1;

  const uint32_t M = rows.end;
  const uint32_t G = K / kGroup;
  const uint32_t nb = n0 / kGroup;

  const __amdgpu_buffer_rsrc_t rA = make_rsrc(A, rows.total * K);
  const __amdgpu_buffer_rsrc_t rW = make_rsrc(W, N * K);
  const __amdgpu_buffer_rsrc_t rS = make_rsrc(As, G * Mp * 4);
  const __amdgpu_buffer_rsrc_t rWs = make_rsrc(Ws, ROW ? N * 4 : (N / kGroup) * G * 4);
  // FFN mode: the up weights and their scales
  const __amdgpu_buffer_rsrc_t rW2 = FFN ? make_rsrc(ffn.w_up, N * K) : rW;
  const __amdgpu_buffer_rsrc_t rWs2 = FFN ? make_rsrc(ffn.ws_up, (N / kGroup) * G * 4) : rWs;

  // Operand chunks of this wave (LDS chunk c covers 8 rows of 128 bytes:
  // activations first, then weights; FFN mode: activations 0-15, gate
  // 16-31, up 32-47).  A wave may only overwrite, in its read phase, LDS
  // rows that no other wave of its own group reads:
  //   group 1 (loads in phase A, right after its own reads of block kb):
  //     four chunks that only group 0 reads -- activation rows 0-127 (plain)
  //     or the gate rows (FFN) -- and the scales of itself and of its
  //     group-0 partner wave gw, which only their owners read;
  //   group 0 (loads in phase B, after the phase-A barrier, when both groups
  //     are done with block kb): the other 32 chunks, eight per wave.
  uint32_t c_off[CH0], c_lds[CH0];
  const bool g0_act = !FFN && gw < 2;  // plain group 0: activation rows 128-255 (gw 0, 1) or weights
#pragma unroll
  for (int j = 0; j < CH0; ++j) {
    uint32_t c, ch;  // LDS chunk, chunk within its operand
    bool act;
    if (grp) {
      c = (FFN ? 16 : 0) + 4 * gw + (j & 3);
      ch = 4 * gw + (j & 3);
      act = !FFN;
    } else if constexpr (FFN) {
      c = (j < 4) ? 4 * gw + j : 32 + 4 * gw + (j - 4);
      ch = 4 * gw + (j & 3);
      act = j < 4;
    } else {
      c = 16 + 8 * gw + j;
      ch = g0_act ? c : c - 32;
      act = g0_act;
    }
    const uint32_t row = ch * 8 + (lane >> 3), col = lane & 7;  // row within the operand
    c_lds[j] = c;
    c_off[j] = act ? rows.src(min(m0 + row, M - 1)) * K + (col ^ swz(row)) * 16
                   : (n0 + row) * K + (col ^ swz(row)) * 16;  // swz: low 4 bits of the LDS row
  }
  const uint32_t s_off = rows.scale_slot(m0 + wm * C::WM + lane, Mp) * 4;       // own activation scales
  const uint32_t s_off_p = rows.scale_slot(m0 + (gw >> 1) * C::WM + lane, Mp) * 4;  // partner's (group 1)
  const uint32_t ws_off = nb * G * 4;
  const uint32_t my_sc = C::A_BYTES + C::W_BYTES + wave * C::SCW_BYTES;
  const uint32_t p_sc = C::A_BYTES + C::W_BYTES + gw * C::SCW_BYTES;

  auto issue_g0 = [&](uint32_t kb, uint32_t stage) {
    uint8_t* base = smem + stage * C::STAGE_BYTES;
    unroll_seq(
        [&](auto jc) {
          constexpr int J = decltype(jc)::value;
          if constexpr (FFN)
            dma16(J < 4 ? rA : rW2, c_off[J], kb * kGroup, base + c_lds[J] * 1024);
          else
            dma16(g0_act ? rA : rW, c_off[J], kb * kGroup, base + c_lds[J] * 1024);
        },
        std::make_integer_sequence<int, CH0>{});
  };
  auto issue_g1 = [&](uint32_t kb, uint32_t stage) {
    uint8_t* base = smem + stage * C::STAGE_BYTES;
    unroll_seq(
        [&](auto jc) {
          constexpr int J = decltype(jc)::value;
          dma16(FFN ? rW : rA, c_off[J], kb * kGroup, base + c_lds[J] * 1024);
        },
        std::make_integer_sequence<int, CH1>{});
    dma4(rS, s_off, kb * Mp * 4, base + my_sc);
    dma4(rS, s_off_p, kb * Mp * 4, base + p_sc);
    if constexpr (!ROW) {
      dma4(FFN ? rWs2 : rWs, ws_off, kb * 4, base + my_sc + 256);  // up scales in FFN mode
      dma4(rWs, ws_off, kb * 4, base + p_sc + 256);
    }
  };

  const uint32_t l16 = lane & 15, c0 = 2 * (lane >> 4);
  const uint32_t lo0 = l16 * 128 + ((c0 ^ swz(l16)) * 16);
  const uint32_t lo1 = l16 * 128 + (((c0 + 1) ^ swz(l16)) * 16);
  auto ld16 = [](const uint8_t* p) -> v4i { return *reinterpret_cast<const v4i*>(p); };
  auto ldf = [](const uint8_t* p) -> float { return *reinterpret_cast<const float*>(p); };
  const uint32_t a_row0 = wm * C::WM * 128, w_row0 = C::A_BYTES + wn * C::WN * 128;

  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  v8i af[TM], bf[TN];
  float as[TM], ws = 0.0f, sc[TM], sc_tail = 0.0f;
  v4f p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // read this wave's fragments and scales from LDS slot S (18 LDS reads);
  // the slot is a compile-time constant, so every address is a loop-invariant
  // register plus an immediate offset
  // 16-row sub-tiles of this wave's band that hold rows below M (all TM
  // but in a last row tile that M ends inside; uniform over the wave)
  const uint32_t band0 = m0 + wm * C::WM;
  const uint32_t vt = FFN ? TM : (M <= band0 ? 0u : min((uint32_t)TM, (M - band0 + 15) / 16));
  // read this wave's fragments and scales from LDS slot S (18 LDS reads);
  // the slot is a compile-time constant, so every address is a loop-invariant
  // register plus an immediate offset.  Partial bands (FULL false) skip the
  // activation fragments of sub-tiles past M.
  auto read_block = [&](auto slot_c, auto full_c) {
    const uint8_t* sb = smem + decltype(slot_c)::value * C::STAGE_BYTES;
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) {
      bf[tn].lo = ld16(sb + w_row0 + tn * 2048 + lo0);
      bf[tn].hi = ld16(sb + w_row0 + tn * 2048 + lo1);
    }
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      if (decltype(full_c)::value || (uint32_t)tm < vt) {
        af[tm].lo = ld16(sb + a_row0 + tm * 2048 + lo0);
        af[tm].hi = ld16(sb + a_row0 + tm * 2048 + lo1);
        as[tm] = ldf(sb + my_sc + (tm * 16 + l16) * 4);
      }
    }
    ws = ROW ? 1.0f : ldf(sb + my_sc + 256);
  };
  // MFMAs and promotions of the block in registers; the promotions of its
  // last kPromoteDist MFMAs are left pending for the next block's compute
  // phase.  A partial band runs only the MFMAs of its sub-tiles below M
  // (the others' accumulators hold rows that are never stored): in a last
  // row tile that M ends inside, the group's compute phase shrinks and the
  // matrix pipe spends no power on rows past M.
  auto compute_block = [&](auto full_c) {
    constexpr bool FULL = decltype(full_c)::value;
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) sc[tm] = as[tm] * ws;
    unroll_seq(
        [&](auto ic) {
          constexpr int I = decltype(ic)::value;
          constexpr int tm = I / TN, tn = I % TN;
          if (FULL || (uint32_t)tm < vt) p[I & 3] = mfma_e4m3_128(bf[tn], af[tm]);
          if constexpr (I < kPromoteDist) {
            constexpr int J = NP - kPromoteDist + I;
            if (FULL || (uint32_t)(J / TN) < vt) acc[J / TN][J % TN] += p[J & 3] * sc_tail;
          } else {
            constexpr int J = I - kPromoteDist;
            if (FULL || (uint32_t)(J / TN) < vt) acc[J / TN][J % TN] += p[J & 3] * sc[J / TN];
          }
          sched_fence();
        },
        std::make_integer_sequence<int, NP>{});
    sc_tail = sc[TM - 1];
  };
  using FullT = std::true_type;
  using PartT = std::false_type;

  // Each group runs its own loop (its own body, so no value is live across
  // a merge of the two roles); both execute the same
  // sequence of workgroup barriers.  Every wave issues its part of stages
  // 0 .. STAGES-1 up front and its part of stage kb+STAGES (slot kb %
  // STAGES) in its read phase of iteration kb: group 1 in phase A, after its
  // own reads of block kb, only rows that group 0 alone reads (group 0 read
  // them one phase earlier); group 0 in phase B, after the phase-A barrier,
  // when both groups are done with block kb.  (A group-1 load of rows that
  // another group-1 wave reads could overwrite them before that wave has
  // read them: the direct loads land within a few hundred cycles when the
  // operands sit in L2.)
  // The K loop is unrolled by STAGES so that each copy's slot (kb % STAGES)
  // is a compile-time constant.
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  using S2 = std::integral_constant<int, 2>;
  static_assert(STAGES == 3, "the unrolled loop below assumes three slots");
  if (grp == 0) {
    // iteration kb: phase A computes block kb, phase B reads block kb+1
    // (block G: a reloaded copy of the last block, unused) and refills slot
    // kb % STAGES with block kb+STAGES
    auto run = [&](auto full_c) {
      auto step = [&](uint32_t kb, auto slot_c) {
        constexpr int S = decltype(slot_c)::value;
        compute_block(full_c);  // phase A
        wait_vmcnt<LW0>();      // own part of stage kb+1 (that of kb+2 may be in flight)
        wg_barrier();
        read_block(std::integral_constant<int, (S + 1) % STAGES>{}, full_c);  // phase B
        wait_lgkm0();
        issue_g0(min(kb + STAGES, G - 1), S);
        wg_barrier();
      };
#pragma unroll
      for (int s = 0; s < STAGES; ++s) issue_g0(min((uint32_t)s, G - 1), s);
      wait_vmcnt<(STAGES - 1) * LW0>();  // own part of stage 0
      wg_barrier();
      read_block(S0{}, full_c);
      wait_lgkm0();
      wg_barrier();
      uint32_t kb = 0;
      for (; kb + 3 <= G; kb += 3) {
        step(kb, S0{});
        step(kb + 1, S1{});
        step(kb + 2, S2{});
      }
      if (kb < G) step(kb, S0{});
      if (kb + 1 < G) step(kb + 1, S1{});
    };
    if (vt == (uint32_t)TM)
      run(FullT{});
    else
      run(PartT{});
  } else {
    // iteration kb: phase A reads block kb and refills its slot, phase B
    // computes it
    auto run = [&](auto full_c) {
      auto step = [&](uint32_t kb, auto slot_c) {
        constexpr int S = decltype(slot_c)::value;
        read_block(slot_c, full_c);  // phase A
        wait_lgkm0();
        issue_g1(min(kb + STAGES, G - 1), S);
        wait_vmcnt<2 * LW1>();  // own part of stage kb+1 (kb+2, kb+3 may be in flight)
        wg_barrier();
        compute_block(full_c);  // phase B
        wg_barrier();
      };
#pragma unroll
      for (int s = 0; s < STAGES; ++s) issue_g1(min((uint32_t)s, G - 1), s);
      wait_vmcnt<(STAGES - 1) * LW1>();  // own part of stage 0
      wg_barrier();
      wg_barrier();
      uint32_t kb = 0;
      for (; kb + 3 <= G; kb += 3) {
        step(kb, S0{});
        step(kb + 1, S1{});
        step(kb + 2, S2{});
      }
      if (kb < G) step(kb, S0{});
      if (kb + 1 < G) step(kb + 1, S1{});
    };
    if (vt == (uint32_t)TM)
      run(FullT{});
    else
      run(PartT{});
  }
  wait_vmcnt<0>();  // no direct load may still be writing LDS at exit
#pragma unroll
  for (int j = NP - kPromoteDist; j < NP; ++j) acc[j / TN][j % TN] += p[j & 3] * sc_tail;
  if constexpr (FFN) {
    ffn_epilogue<TM, TN>(acc, smem, ffn, wave, lane, m0 + wm * C::WM, n0 + (wn & 1) * C::WN, nb,
                         M, N, rows.pad_end(Mp));
    return;
  }
  if constexpr (ROW) {
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) {
      const float4 r = *reinterpret_cast<const float4*>(Ws + n0 + wn * C::WN + tn * 16 + 4 * (lane >> 4));
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) acc[tm][tn] *= v4f{r.x, r.y, r.z, r.w};
    }
  }

  epi.template add<TM, TN, C::NT, C::BM>([&](int tm, int tn) -> v4f& { return acc[tm][tn]; }, smem, m0,
                                         wm * C::WM, n0 + wn * C::WN, M, lane, 0);
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const uint32_t m = m0 + wm * C::WM + tm * 16 + l16;
    if (m < M) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        const uint32_t n = n0 + wn * C::WN + tn * 16 + 4 * (lane >> 4);
        *reinterpret_cast<uint2*>(out + (uint64_t)m * N + n) = pack_bf16x4(acc[tm][tn]);
      }
    }
  }
}

}  // namespace
}  // namespace fp8q
