// The LDS-tiled block-scaled FP8 GEMM: tile geometry and the kernel body, shared
// by the dense kernels (gemm.hip), the expert-grouped ones (grouped.hip) and
// the projection with per-request adapters (lora.hip).
#pragma once

#include "gemm_rows.h"
#include "mfma_common.h"

namespace fp8q {
namespace {

// Promotion distance: the fp32 promotion of MFMA i is issued in the slot of
// MFMA i + kPromoteDist.  A VALU read of an MFMA result waits until the
// matrix pipe has written it; measured with one wave per SIMD issuing
// 16x16x128 FP8 MFMAs and four promotion fmas per MFMA from registers, the
// matrix pipe is busy 51% / 75% / 91% of the time at distance 1 / 2 / 3
// (99% without the fmas).  The results rotate through four register sets,
// so the distance is at most 3, and the last kPromoteDist MFMAs of a K block
// (promoted in the next block, with that block's scale) lie in one row.
constexpr int kPromoteDist = 3;

__device__ __forceinline__ v4f mfma_e4m3_128(const v8i& w, const v8i& a) {
  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  // cbsz = blgp = 0: both operands OCP e4m3; zero scale operands select the
  // unscaled instruction.
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, zero, 0, 0, 0, 0, 0, 0);
}

// ------------------------------------------------------------------------
// LDS-tiled kernel.  Workgroup tile BM x BN, K step 128 (one scale block),
// WGM x WGN waves, each owning a WM x WN = (BM/WGM) x (BN/WGN) sub-tile made
// of TM x TN MFMA tiles of 16 x 16.
//
// Operands reach LDS through direct buffer->LDS loads (64 lanes x 16 B land in
// 1 KB of consecutive LDS), so the ring of STAGES LDS buffers is filled
// without staging registers.  A stage holds [BM rows][128 B] of activations,
// [BN rows][128 B] of weights and, per wave, the activation scales of its WM
// rows (read from the K-major scale layout, where they are contiguous) and 64
// copies of the block's weight scale.  16-byte chunk c of row r sits at chunk
// position c ^ f(r), f(r) = (r & 7) ^ ((r >> 3) & 1), so the 16 lanes that
// read one chunk column of 16 consecutive rows hit 16 different (row parity,
// chunk) bank groups; f depends on r mod 16 only, so every fragment address is
// a per-lane constant plus a compile-time offset.  The direct load realises
// the swizzle by choosing, per lane, which global chunk lands in its fixed
// LDS slot.
//
// Register pipeline, per K block: the MFMAs of block kb run from registers
// while the fragments of block kb+1 are read from LDS into a second register
// set (activation fragments in place, as soon as the last MFMA of their row
// has been issued).  The fp32 promotion of MFMA i is issued after MFMA
// i + kPromoteDist, by which time the matrix pipe has written its result; the
// promotions of a block's last kPromoteDist MFMAs run in the next block.
// Each MFMA slot (the MFMA, the four fmas, one or two LDS reads) is fenced
// off from the next with a scheduling barrier: left to itself the compiler hoists all MFMAs of a block and then
// has to serialise the next one on a single result register.
// ------------------------------------------------------------------------
template <int BM, int BN, int WGM, int WGN, int STAGES, bool ROW = false>
struct TileCfg {
  static constexpr int NW = WGM * WGN, NT = 64 * NW;
  static constexpr int WM = BM / WGM, WN = BN / WGN, TM = WM / 16, TN = WN / 16, NP = TM * TN;
  static constexpr int A_BYTES = BM * 128, W_BYTES = BN * 128;
  static constexpr int SA = (WM + 63) / 64;        // activation-scale loads per wave and stage
  static constexpr int SCW_BYTES = SA * 256 + 256;  // per wave: its scales + 64 weight-scale copies
  static constexpr int STAGE_BYTES = A_BYTES + W_BYTES + NW * SCW_BYTES;
  static constexpr int LDS_BYTES = STAGES * STAGE_BYTES;
  static constexpr int DA = BM * 8 / 64 / NW;  // 1 KB direct loads per wave: activations
  static constexpr int DW = BN * 8 / 64 / NW;  //                              weights
  static constexpr int LOADS = DA + DW + SA + (ROW ? 0 : 1);  // direct loads per wave and stage
  // LDS reads of the next block per MFMA slot: slot TN*tm + TN-1 (after the
  // last MFMA of row tm) reads activation fragment tm; the other slots take,
  // in order, the 2*TN weight-fragment halves, TM/2 activation-scale pairs
  // and the weight scale.
  static constexpr int FREE_OPS = 2 * TN + TM / 2 + (ROW ? 0 : 1);
  static_assert(WM % 16 == 0 && WN % 16 == 0 && TN >= 2 && TM % 2 == 0 && NP % 4 == 0, "wave tile");
  static_assert(NP - TM >= FREE_OPS, "too few MFMA slots for the LDS reads");
  static_assert(kPromoteDist >= 1 && kPromoteDist <= 3 && kPromoteDist <= TN && NP % 4 == 0,
                "pending promotions lie in the last row; four result registers");
  static_assert(BM * 8 % (64 * NW) == 0 && BN * 8 % (64 * NW) == 0, "tile/wave mismatch");
  static_assert(128 % WN == 0, "a wave's columns lie in one weight-scale block");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS budget");
  static_assert(STAGES >= 2 && (STAGES - 2) * LOADS < 64, "vmcnt range");
  static_assert(STAGE_BYTES % 256 == 0, "stage alignment");
};

// ROW: per-row weight scales Ws[N] (one multiplier per output column,
// applied to the finished accumulator) instead of 128x128 block scales
// applied per K block.
//
// SPLIT: split-K.  The grid holds `splits` workgroups per tile; split s takes
// the K blocks [s*G/splits, (s+1)*G/splits) and stores its fp32 partial tile
// to part[s][M][N]; a second kernel (splitk_reduce_kernel) adds the splits'
// partials in split order and rounds to bf16.  Block-scaled weights only.
//
// Rows (gemm_rows.h) says which activation rows a tile's output rows read and
// where its rows end; Epi adds to the finished accumulators before the store
// (NoEpilogue: nothing).  The tile is rows m0.. and columns n0.. .
template <int BM, int BN, int WGM, int WGN, int STAGES, bool ROW, bool SPLIT, class Rows, class Epi,
          int WAUX = 0>
__device__ __forceinline__ void gemm_tiled_body(
    const uint8_t* __restrict__ A, const float* __restrict__ As, const uint8_t* __restrict__ W,
    const float* __restrict__ Ws, uint16_t* __restrict__ out, uint32_t m0, uint32_t n0, uint32_t N,
    uint32_t K, uint32_t Mp, uint32_t split, uint32_t splits, float* __restrict__ part,
    const Rows& rows, const Epi& epi) {
  using C = TileCfg<BM, BN, WGM, WGN, STAGES, ROW>;
  constexpr int TM = C::TM, TN = C::TN, NP = C::NP;
  static_assert(!(SPLIT && ROW), "split-K for block-scaled weights only");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];

  const uint32_t tid = threadIdx.x, lane = tid & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // wave-uniform (SGPR)
  const uint32_t wm = wave / WGN, wn = wave % WGN;

  const uint32_t M = rows.end;
  const uint32_t GK = K / kGroup;  // K blocks in all
  // this workgroup's K blocks: kbeg .. kbeg + G - 1
  const uint32_t kbeg = SPLIT ? split * GK / splits : 0;
  const uint32_t G = SPLIT ? (split + 1) * GK / splits - kbeg : GK;
  const uint32_t nb = (n0 + wn * C::WN) / kGroup;  // this wave's weight-scale block row

  // ---- buffer resources and per-lane source offsets (K block 0) ----
  const __amdgpu_buffer_rsrc_t rA = make_rsrc(A, rows.total * K);
  const __amdgpu_buffer_rsrc_t rW = make_rsrc(W, N * K);
  const __amdgpu_buffer_rsrc_t rS = make_rsrc(As, GK * Mp * 4);
  const __amdgpu_buffer_rsrc_t rWs = make_rsrc(Ws, ROW ? N * 4 : (N / kGroup) * GK * 4);
  uint32_t a_off[C::DA], w_off[C::DW], s_off[C::SA];
#pragma unroll
  for (int j = 0; j < C::DA; ++j) {
    const uint32_t c = (wave * C::DA + j) * 64 + lane, row = c >> 3;
    a_off[j] = rows.src(min(m0 + row, M - 1)) * K + ((c & 7) ^ swz(row)) * 16;
  }
#pragma unroll
  for (int j = 0; j < C::DW; ++j) {
    const uint32_t c = (wave * C::DW + j) * 64 + lane, row = c >> 3;
    w_off[j] = (n0 + row) * K + ((c & 7) ^ swz(row)) * 16;
  }
  // activation scales of this wave's rows (rows past Mp are clamped in
  // bounds and never used; rows in [M, Mp) hold the layout's zero pad)
#pragma unroll
  for (int j = 0; j < C::SA; ++j) s_off[j] = rows.scale_slot(m0 + wm * C::WM + j * 64 + lane, Mp) * 4;
  const uint32_t ws_off = nb * GK * 4;  // every lane loads the same weight scale
  const uint32_t sc_base = C::A_BYTES + C::W_BYTES + wave * C::SCW_BYTES;
  const uint32_t ws_base = sc_base + C::SA * 256;

  // K block kbeg + kl (kl counted from this workgroup's first block)
  auto issue_stage = [&](uint32_t kl, uint32_t stage) {
    const uint32_t kb = kbeg + kl;
    uint8_t* base = smem + stage * C::STAGE_BYTES;
#pragma unroll
    for (int j = 0; j < C::DA; ++j) dma16(rA, a_off[j], kb * kGroup, base + (wave * C::DA + j) * 1024);
#pragma unroll
    for (int j = 0; j < C::DW; ++j)
      dma16_aux<WAUX>(rW, w_off[j], kb * kGroup, base + C::A_BYTES + (wave * C::DW + j) * 1024);
#pragma unroll
    for (int j = 0; j < C::SA; ++j) dma4(rS, s_off[j], kb * Mp * 4, base + sc_base + j * 256);
    if constexpr (!ROW) dma4(rWs, ws_off, kb * 4, base + ws_base);
  };

  // Per-lane byte offsets of a fragment inside a 16-row slab: this lane's row
  // (lane % 16) and its two chunks 2*(lane/16) and 2*(lane/16)+1, swizzled.
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

  // ---- prologue: the first STAGES stages, then block 0 into registers ----
  // Stages past the last K block reload the last block (in bounds, never
  // read), so that every iteration issues the same loads and waits for the
  // same count, and the loop body stays one basic block per K block.
#pragma unroll
  for (int s = 0; s < STAGES; ++s) issue_stage(min((uint32_t)s, G - 1), s);
  wait_vmcnt<(STAGES - 1) * C::LOADS>();
  wg_barrier();

  v8i af[TM], bf0[TN], bf1[TN];
  float as0[TM], as1[TM], ws0, ws1;
  {
    const uint8_t* s0 = smem;  // slot 0
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      af[tm].lo = ld16(s0 + a_row0 + tm * 2048 + lo0);
      af[tm].hi = ld16(s0 + a_row0 + tm * 2048 + lo1);
      as0[tm] = ldf(s0 + sc_base + (tm * 16 + l16) * 4);
    }
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) {
      bf0[tn].lo = ld16(s0 + w_row0 + tn * 2048 + lo0);
      bf0[tn].hi = ld16(s0 + w_row0 + tn * 2048 + lo1);
    }
    ws0 = ROW ? 1.0f : ldf(s0 + ws_base);
  }
  ws1 = 1.0f;

  // MFMA results rotate through 4 register sets; the promotions of the last
  // kPromoteDist MFMAs of a block are pending when the next block starts
  // (zero before the first block).
  v4f p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  float sc[TM], sc_tail = 0.0f;

  // one K block; S = kb % STAGES, a compile-time constant (the loop below is
  // unrolled by a multiple of STAGES), so that the LDS addresses of the next
  // block's fragments are loop-invariant registers plus immediate offsets
  auto step = [&](uint32_t kb, auto slot_c, const v8i(&bf)[TN], const float(&as)[TM], float ws,
                  v8i(&bfn)[TN], float(&asn)[TM], float& wsn) {
    constexpr int S = decltype(slot_c)::value;
    wait_lgkm0();  // fragments and scales of block kb are in registers
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) sc[tm] = as[tm] * ws;
    wait_vmcnt<(STAGES - 2) * C::LOADS>();
    wg_barrier();  // stage kb+1 is in LDS; slot kb % STAGES is free
    issue_stage(min(kb + STAGES, G - 1), S);
    // (on the last block the reads below fetch a slot holding a reloaded
    // copy of the last block, never used; its load has completed)
    const uint8_t* nx = smem + ((S + 1) % STAGES) * C::STAGE_BYTES;
    unroll_seq(
        [&](auto ic) {
          constexpr int I = decltype(ic)::value;
          constexpr int tm = I / TN, tn = I % TN;
          p[I & 3] = mfma_e4m3_128(bf[tn], af[tm]);
          if constexpr (I < kPromoteDist) {
            constexpr int J = NP - kPromoteDist + I;
            acc[J / TN][J % TN] += p[J & 3] * sc_tail;
          } else {
            constexpr int J = I - kPromoteDist;
            acc[J / TN][J % TN] += p[J & 3] * sc[J / TN];
          }
          if constexpr (tn == TN - 1) {
            af[tm].lo = ld16(nx + a_row0 + tm * 2048 + lo0);
            af[tm].hi = ld16(nx + a_row0 + tm * 2048 + lo1);
          } else {
            constexpr int Q = I - I / TN;
            if constexpr (Q < 2 * TN) {
              if constexpr (Q & 1) bfn[Q / 2].hi = ld16(nx + w_row0 + (Q / 2) * 2048 + lo1);
              else bfn[Q / 2].lo = ld16(nx + w_row0 + (Q / 2) * 2048 + lo0);
            } else if constexpr (Q < 2 * TN + TM / 2) {
              constexpr int T2 = 2 * (Q - 2 * TN);
              asn[T2] = ldf(nx + sc_base + (T2 * 16 + l16) * 4);
              asn[T2 + 1] = ldf(nx + sc_base + ((T2 + 1) * 16 + l16) * 4);
            } else if constexpr (!ROW && Q == 2 * TN + TM / 2) {
              wsn = ldf(nx + ws_base);
            }
          }
          sched_fence();
        },
        std::make_integer_sequence<int, NP>{});
    sc_tail = sc[TM - 1];
  };
  // block kb0 + I: register set I % 2, LDS slot I % STAGES
  auto step_i = [&](uint32_t kb0, auto ic) {
    constexpr int I = decltype(ic)::value;
    using Slot = std::integral_constant<int, I % STAGES>;
    if constexpr (I % 2 == 0)
      step(kb0 + I, Slot{}, bf0, as0, ws0, bf1, as1, ws1);
    else
      step(kb0 + I, Slot{}, bf1, as1, ws1, bf0, as0, ws0);
  };
  constexpr int U = STAGES % 2 == 0 ? STAGES : 2 * STAGES;  // blocks per loop iteration
  uint32_t kb = 0;
  for (; kb + U <= G; kb += U)
    unroll_seq([&](auto ic) { step_i(kb, ic); }, std::make_integer_sequence<int, U>{});
  unroll_seq(
      [&](auto ic) {
        if (kb + decltype(ic)::value < G) step_i(kb, ic);
      },
      std::make_integer_sequence<int, U - 1>{});
  wait_vmcnt<0>();  // no direct load may still be writing LDS when the workgroup ends
  // promotions of the last block's last kPromoteDist MFMAs (all in its last row)
#pragma unroll
  for (int j = NP - kPromoteDist; j < NP; ++j) acc[j / TN][j % TN] += p[j & 3] * sc_tail;

  if constexpr (ROW) {
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) {
      const float4 r = *reinterpret_cast<const float4*>(Ws + n0 + wn * C::WN + tn * 16 + 4 * (lane >> 4));
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) acc[tm][tn] *= v4f{r.x, r.y, r.z, r.w};
    }
  }
  epi.template add<TM, TN, C::NT, BM>([&](int tm, int tn) -> v4f& { return acc[tm][tn]; }, smem, m0, wm * C::WM,
                                      n0 + wn * C::WN, M, lane, SPLIT ? split : 0);
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const uint32_t m = m0 + wm * C::WM + tm * 16 + (lane & 15);
    if (m < M) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        const uint32_t n = n0 + wn * C::WN + tn * 16 + 4 * (lane >> 4);
        if constexpr (SPLIT)
          *reinterpret_cast<v4f*>(part + ((uint64_t)split * rows.total + m) * N + n) = acc[tm][tn];
        else
          *reinterpret_cast<uint2*>(out + (uint64_t)m * N + n) = pack_bf16x4(acc[tm][tn]);
      }
    }
  }
}

}  // namespace
}  // namespace fp8q
