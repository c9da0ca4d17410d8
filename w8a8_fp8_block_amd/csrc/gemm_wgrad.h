// The weights' gradient dw[n,k] = sum over tokens m of dy[m,n] * x[m,k], both
// operands FP8 with one power of two per column and 128 tokens, both in their own
// row-major layout.
//
//   dw[n,k] = sum_b 2^(ey[b,n] + ex[b,k]) * sum_{m in block b} dec(dy[m,n]) * dec(x[m,k])
//
// The sum runs along the rows of both matrices, so their fragments come through
// the transposing LDS read (gemm_grad.h) and no transposed copy exists.  The
// scales are the matrix instruction's own operands, a byte a lane: the partial
// products need no fp32 multiply of their own and add up in the instruction's fp32
// accumulators over all the tokens.  As exact as scaled fp32 additions: 1.5e-5 of the
// result's norm either way over 4608 tokens, and the same over 65536 (2.6e-6 for products
// of one sign); it is the instruction's rounding of its 64 products that shows.
//
// Pipeline.  A workgroup of four waves computes a tile of BM = 64 TM columns of dy
// by BN = 64 TN columns of x, its waves in a 2 x 2 grid.  The tokens pass in halves
// of a block, 64 at a time, through a ring of SLOTS LDS slots filled by direct loads:
// [panel of 128 columns][64 tokens][128 bytes], then the columns' scale dwords.  Of
// each half a wave holds its TM + TN fragments in registers, read while the products
// of the half before it run: one set of fragments per parity, one barrier a half.
// The reads, the direct loads and the barrier lie between matrix instructions, each
// in the shadow of one (64 cycles); left in a row at the start of a half, the loads
// alone cost 10%.
//
// LDS bounds the tile: a wave of 64 x 64 reads 8 KB for 256 cycles of matrix
// instructions, 32 bytes a cycle, and four SIMDs of them the 128 that LDS delivers,
// with the direct loads' writes to come; at 128 x 128 it is half of that.  That
// takes 256 accumulators a lane, so one wave a SIMD, which issues instructions of all
// kinds by itself.  (Two waves of 128 x 64 a SIMD: 2634 TFLOP/s over 4096 x 4096 x
// 18304 tokens against 2800; the same two taking turns between reading and computing:
// 2546.  A library's FP8 product with one scale for all, 8192^3: 2642.)
//
// 4576 x 17408 x 5120: 314-327 us by card, 2.5-2.6 PFLOP/s, at that library product's rate;
// 409 x 2048 x 1408: 5.8 us.
//
// The direct loads are issued in assembly (gemm_grad.h says why: the waits that the
// compiler would add cost half the speed).
//
// Fragments of 32 columns x 64 tokens: lane l holds column l % 32, tokens
// 32 (l / 32) ..; the transposing read takes chunk 2 t + (l / 16) % 2 of the panel for
// the 16 lanes of l's row.  Tokens past M lie past the buffer resources' ends and
// load as zeros.
#pragma once

#include "gemm_grad.h"

namespace fp8q {
namespace {

struct WgradArgs {
  const uint8_t *dy, *x;     // codes [M,N], [M,K]
  const uint32_t *ey, *ex;   // [ceil(M/512)][N], [K]: four token blocks' bytes a dword
  uint16_t* out;             // [N,K] bf16
  float* part;               // split form: [splits][N][K]
  uint32_t M, N, K, tiles_n, tiles_k, splits;
};

template <int TM_, int TN_>
struct WgradCfg {
  static constexpr int TM = TM_, TN = TN_, SLOTS = 4;
  static constexpr int BM = 64 * TM, BN = 64 * TN;  // 2 x 2 waves of TM x TN 32 x 32 tiles
  static constexpr int PY = BM / 128, PX = BN / 128, PANELS = (BM + BN) / 128, PANEL = 64 * 128;
  static constexpr int SC = PANELS * PANEL;  // the scales' place in a slot: 512 bytes a panel
  static constexpr int SLOT_BYTES = SC + PANELS * 512, LDS_BYTES = SLOTS * SLOT_BYTES;
  // loads of a wave and half: two 1 KB chunks (8 rows) of each panel, and 256 bytes of
  // each operand's scales (with one panel two waves load the same)
  static constexpr int CH = 2 * PANELS, LOADS = CH + 2;
  static constexpr int OPS = 3 * (TM + TN);          // LDS reads of a half: fragment halves, scales
  // where in the half's TM * TN products the barrier and the reads lie, and how far behind
  // the barrier the loads begin
  static constexpr int BAR = TM * TN >= 8 ? 1 : 0, READS_END = TM * TN - (TM * TN >= 8 ? 3 : 0);
  static constexpr int LOADS_FROM = TM * TN >= 16 ? 2 : 0;
  static_assert(BM % 128 == 0 && BN % 128 == 0 && LDS_BYTES <= 160 * 1024, "tile");
  static_assert((SLOTS - 1) * LOADS < 64, "vmcnt range");
};

// Quads of halves (two token blocks; one round of the ring) that `blocks` blocks take.
__device__ __forceinline__ uint32_t wgrad_quads(uint32_t blocks) { return (blocks + 1) / 2; }

// The tiles next(u) -> (n0, k0), u = 0 .. units - 1, one after the other, each over the
// tokens m0 .. m1 - 1 (m0 a multiple of 128, m0 < m1, units > 0).  The ring runs on from
// one tile into the next, so a tile's stores lie over the next one's loads.
template <class C, bool SPLIT, class Next>
__device__ __forceinline__ void gemm_wgrad_body(const WgradArgs& a, uint32_t units, uint32_t m0, uint32_t m1,
                                                uint32_t split, const Next& next) {
  constexpr int TM = C::TM, TN = C::TN, SLOTS = C::SLOTS;
  static_assert(SLOTS == 4, "a quad of halves is one round of the ring");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t wm = wave >> 1, wn = wave & 1;
  const uint32_t N = a.N, K = a.K, packs = (a.M + 511) / 512;
  const uint32_t Q = wgrad_quads((m1 - m0 + 127) / 128), h_end = (m1 + 63) / 64;

  // ---- loads: a quad ahead of the products ----
  // Wave w's chunks of a panel hold its rows 16 w + 8 j ..; row r's 16-byte chunk p lies
  // at p ^ swz_t(r).  The resources start at the tile's first column.
  const uint32_t lrow = lane >> 3, lcol = ((lane & 7) ^ lrow ^ (wave >> 1)) * 16;
  const uint32_t y_off[2] = {(16 * wave + lrow) * N + lcol, (16 * wave + lrow + 8) * N + lcol};
  const uint32_t x_off[2] = {(16 * wave + lrow) * K + lcol, (16 * wave + lrow + 8) * K + lcol};
  const uint32_t sc_y = wave % (2 * C::PY) * 256, sc_x = wave % (2 * C::PX) * 256;
  const uint32_t ey_off = sc_y + lane * 4, ex_off = sc_x + lane * 4;
  const uint32_t lds_w = lds_addr(smem) + wave * 2048;
  const uint32_t lds_ey = lds_addr(smem) + C::SC + sc_y, lds_ex = lds_addr(smem) + C::SC + C::PY * 512 + sc_x;
  u32x4s rY, rX, rEy, rEx;
  uint32_t lh = m0 / 64;  // the quad's first half
  auto aim_tile = [&](bool some, uint32_t n0, uint32_t k0) {
    rY = rsrc_words(a.dy + n0, some ? m1 * N - n0 : 0);
    rX = rsrc_words(a.x + k0, some ? m1 * K - k0 : 0);
    rEy = rsrc_words(a.ey + n0, some ? (packs * N - n0) * 4 : 0);
    rEx = rsrc_words(a.ex + k0, some ? (packs * K - k0) * 4 : 0);
  };
  // Load J of the quad's half S.  Past the last token (or tile) the base is the bound, which
  // leaves nothing before it: zeros, no traffic.  (A base past the bound would leave
  // everything: the bound less the base is what offsets are held against.)
  auto load_op = [&](auto sc, auto jc) {
    constexpr uint32_t S = decltype(sc)::value, J = decltype(jc)::value, P = J / 2;
    constexpr int SLOT = S * C::SLOT_BYTES;
    if constexpr (J < 2u * C::PY)
      dma16_asm<P * 128, SLOT + P * C::PANEL + J % 2 * 1024>(
          rY, y_off[J % 2], min(min(lh + S, h_end) * 64 * N, rY[2]), lds_w);
    else if constexpr (J < (uint32_t)C::CH)
      dma16_asm<(P - C::PY) * 128, SLOT + P * C::PANEL + J % 2 * 1024>(
          rX, x_off[J % 2], min(min(lh + S, h_end) * 64 * K, rX[2]), lds_w);
    else if constexpr (J == (uint32_t)C::CH)
      dma4_asm<SLOT>(rEy, ey_off, min(((lh + S) >> 3) * N * 4, rEy[2]), lds_ey);
    else
      dma4_asm<SLOT>(rEx, ex_off, min(((lh + S) >> 3) * K * 4, rEx[2]), lds_ex);
  };

  // ---- fragments ----
  const uint32_t l32 = lane & 31, row = 32 * (lane >> 5) + ((lane & 15) >> 1);
  const uint32_t lt = row * 128 + (swz_t(row) ^ ((lane >> 4) & 1)) * 16 + (lane & 1) * 8;
  const uint32_t sy = C::SC + (wm * 32 * TM + l32) * 4, sx = C::SC + C::PY * 512 + (wn * 32 * TN + l32) * 4;
  uint32_t ly[TM], lx[TN];
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const uint32_t col = wm * 32 * TM + t * 32;
    ly[t] = col / 128 * C::PANEL + (lt ^ (col % 128));
  }
#pragma unroll
  for (int t = 0; t < TN; ++t) {
    const uint32_t col = wn * 32 * TN + t * 32;
    lx[t] = (C::PY + col / 128) * C::PANEL + (lt ^ (col % 128));
  }
  v8i fy[2][TM], fx[2][TN];
  uint32_t ey[2][TM], ex[2][TN];
  auto read_op = [&](const uint8_t* base, auto set_c, auto q_c) {
    constexpr int S = decltype(set_c)::value, O = decltype(q_c)::value;
    if constexpr (O < 2 * TN) {
      if constexpr (O & 1) fx[S][O / 2].hi = ld_transposed(base + lx[O / 2], 1);
      else fx[S][O / 2].lo = ld_transposed(base + lx[O / 2], 0);
    } else if constexpr (O < 2 * TN + 2 * TM) {
      constexpr int P = O - 2 * TN;
      if constexpr (P & 1) fy[S][P / 2].hi = ld_transposed(base + ly[P / 2], 1);
      else fy[S][P / 2].lo = ld_transposed(base + ly[P / 2], 0);
    } else if constexpr (O < 2 * TN + 3 * TM) {
      constexpr int P = O - 2 * TN - 2 * TM;
      ey[S][P] = *reinterpret_cast<const uint32_t*>(base + sy + P * 128);
    } else {
      constexpr int P = O - 2 * TN - 3 * TM;
      ex[S][P] = *reinterpret_cast<const uint32_t*>(base + sx + P * 128);
    }
  };

  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  uint32_t n0, k0;
  next(0, n0, k0);
  aim_tile(true, n0, k0);
  unroll_seq(
      [&](auto s) { unroll_seq([&](auto j) { load_op(s, j); }, std::make_integer_sequence<int, C::LOADS>{}); },
      std::make_integer_sequence<int, SLOTS>{});
  wait_vmcnt<(SLOTS - 1) * C::LOADS>();
  wg_barrier();
  unroll_seq([&](auto q) { read_op(smem, std::integral_constant<int, 0>{}, q); },
             std::make_integer_sequence<int, C::OPS>{});

  // Products of the quad's half S, whose fragments are in set S % 2; the next half's
  // fragments into the other set, half S of the next quad into the slot.
  uint32_t sh0 = 0;  // the place of the quad's first scale byte
  auto step = [&](auto sc) {
    constexpr int S = decltype(sc)::value, F = S & 1;
    const uint8_t* nx = smem + (S + 1) % SLOTS * C::SLOT_BYTES;
    const uint32_t sh = (sh0 + S / 2 * 8) & 31;
    wait_lgkm0();  // this half's fragments are in registers
#pragma unroll
    for (int t = 0; t < TM; ++t) ey[F][t] >>= sh;
#pragma unroll
    for (int t = 0; t < TN; ++t) ex[F][t] >>= sh;
    sched_fence();
    unroll_seq(
        [&](auto ic) {
          constexpr int I = decltype(ic)::value, P = TM * TN;
          if constexpr (I == C::BAR) {
            // the next half has landed (two more halves' loads are younger, and a tile's
            // stores, which only make the wait longer); every wave has read this half's slot
            wait_vmcnt<(SLOTS - 2) * C::LOADS>();
            sched_fence();
            wg_barrier();
            sched_fence();
          }
          acc[I / TN][I % TN] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              fx[F][I % TN], fy[F][I / TN], acc[I / TN][I % TN], 0, 0, 0, (int)ex[F][I % TN], 0, (int)ey[F][I / TN]);
          if constexpr (I >= C::BAR) {
            constexpr int R = I - C::BAR, RN = C::READS_END - C::BAR;
            if constexpr (R < RN) {
              constexpr int O0 = R * C::OPS / RN, O1 = (R + 1) * C::OPS / RN;
              unroll_seq([&](auto q) { read_op(nx, std::integral_constant<int, 1 - F>{},
                                               std::integral_constant<int, O0 + decltype(q)::value>{}); },
                         std::make_integer_sequence<int, O1 - O0>{});
            }
            constexpr int L = R - C::LOADS_FROM, LN = P - C::BAR - C::LOADS_FROM;
            if constexpr (L >= 0) {
              constexpr int J0 = L * C::LOADS / LN, J1 = (L + 1) * C::LOADS / LN;
              unroll_seq([&](auto j) { load_op(sc, std::integral_constant<int, J0 + decltype(j)::value>{}); },
                         std::make_integer_sequence<int, J1 - J0>{});
            }
          }
          sched_fence();
        },
        std::make_integer_sequence<int, TM * TN>{});
  };
#pragma unroll 1
  for (uint32_t u = 0;;) {
    // The loads' aim changes between quads only: a branch among a quad's products, and the
    // compiler moves them behind it.
    uint32_t nn0 = 0, nk0 = 0;
#pragma unroll 1
    for (uint32_t q = 0; q < Q; ++q) {
      sh0 = (8 * (m0 / 128) + 16 * q) & 31;
      if (q + 1 < Q) {
        lh += 4;
      } else {
        lh = m0 / 64;
        if (u + 1 < units) next(u + 1, nn0, nk0);
        aim_tile(u + 1 < units, nn0, nk0);
      }
      unroll_seq([&](auto s) { step(s); }, std::make_integer_sequence<int, SLOTS>{});
    }
    // N and K are multiples of 128: a wave's share lies inside whole or not at all.  Lane:
    // row n = 32 i + l32, columns k = 32 j + 8 (r / 4) + 4 (lane / 32) + r % 4.  A row
    // group's place is uniform, the lane's within it (at) below 2^32 bytes.
    const bool inside = n0 + wm * 32 * TM < N && k0 + wn * 32 * TN < K;
    sched_fence();
    const uint32_t at = SPLIT ? l32 * K * 4 + 16 * (lane >> 5)
                              : (lane & 15) * K * 2 + 32 * ((lane >> 4) & 1) + 16 * (lane >> 5);
    const uint64_t corner = (uint64_t)(n0 + wm * 32 * TM) * K + (k0 + wn * 32 * TN);
    const uint64_t base = SPLIT ? (uint64_t)(a.part + (uint64_t)split * N * K + corner) : (uint64_t)(a.out + corner);
    if constexpr (SPLIT) {
      // The stores below read the matrix instructions' results in assembly, for which the
      // compiler keeps no wait states: 20 behind the last one's 16 passes.
      asm volatile("s_nop 15\n\ts_nop 3" ::: "memory");
      sched_fence();
    }
    if (inside) {
      unroll_seq(
          [&](auto ic) {
            constexpr int i = decltype(ic)::value / TN, j = decltype(ic)::value % TN;
            const v16f& c = acc[i][j];
            const uint64_t band = base + (uint64_t)(32 * i) * K * (SPLIT ? 4 : 2);
            if constexpr (SPLIT) {
              unroll_seq(
                  [&](auto rc) {
                    constexpr int r = 4 * decltype(rc)::value;
                    const v4f v{c[r], c[r + 1], c[r + 2], c[r + 3]};
                    store16_asm<128 * j + 8 * r>(band, at, __builtin_bit_cast(u32x4s, v));
                  },
                  std::make_integer_sequence<int, 4>{});
            } else {
              uint32_t v[2][4];
              tile_rows_bf16(c, v);
              store16_asm<64 * j>(band, at, u32x4s{v[0][0], v[0][1], v[0][2], v[0][3]});
              store16_asm<64 * j>(band + (uint64_t)16 * K * 2, at, u32x4s{v[1][0], v[1][1], v[1][2], v[1][3]});
            }
            sched_fence();  // one tile's accumulators out at a time
          },
          std::make_integer_sequence<int, TM * TN>{});
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    if (++u == units) break;
    n0 = nn0;
    k0 = nk0;
  }
  // no direct load may still be writing LDS when the workgroup ends, or another
  // body's loads begin
  wait_vmcnt<0>();
  wait_lgkm0();
  wg_barrier();
}

}  // namespace
}  // namespace fp8q
