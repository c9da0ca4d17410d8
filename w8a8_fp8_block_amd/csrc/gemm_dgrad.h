// The input's gradient dx[m,k] = sum_n dy[m,n] * w[n,k], one wave a SIMD.
//
//   acc[m,k] += dy_scale[b,m] * w_scale[b,k/128] * sum_{n in block b} dec(dy[m,n]) * dec(w[n,k])
//
// A workgroup of four waves (2 x 2) computes 64 TM rows of dx by 128 columns, each wave
// 32 TM x 64 as TM x 2 tiles of 32 x 32.  A block of the sum, 128 wide, passes through a ring
// of LDS slots filled by direct loads: [rows of dy][128 bytes], [128 rows of w][128 bytes],
// the rows' scales and the block's weight scale.
//
// The fp32 scales forbid accumulating in the matrix instruction: a tile's two instructions
// (halves of the block, 64 cycles each) make its partial product, 16 fmas add it, scaled, to
// the accumulators.  A wave issues instructions of all kinds by itself, so the block is laid
// out over its 4 TM matrix instructions, a slot each: 8 fmas, and the next block's LDS reads,
// the loads of the block SLOTS ahead and the barrier between them.  The fmas of a tile lie a
// slot and more behind its second instruction (right behind it they wait for its result:
// 371 us against 364).  w's fragments have two register sets; dy's are replaced in place once
// their last product is issued, but for the last 32 rows, whose reads would end too late.
//
// 4576 x 17408 x 5120 (256 rows): 350-365 us by card, 2.3 PFLOP/s, the matrix pipes busy
// 61% of the time (69% of a tile's) at 1.8 GHz; 340 with every load from one block, so what is
// left is the issue of one wave, a last round of 208 tiles on 256 CUs and the clock.  The same in 16 x 16 x 128
// instructions with the fmas behind each: 385; the loads in a row at a block's start: 477;
// the loads first and the reads behind a second barrier: 382; eight waves of 64 x 64 in
// turns (gemm_pp.h's loop): 387.
#pragma once

#include "gemm_grad.h"

namespace fp8q {
namespace {

template <int TM_>
struct DgradCfg {
  static constexpr int TM = TM_, TN = 2, NT = TM * TN, SLOTS = TM == 4 ? 3 : 4;
  static constexpr int BM = 64 * TM, BN = 128;
  static constexpr int W_OFF = BM * 128, AS_OFF = W_OFF + 128 * BN, WS_OFF = AS_OFF + BM * 4;
  static constexpr int SLOT_BYTES = WS_OFF + 4 * 256, LDS_BYTES = SLOTS * SLOT_BYTES;
  static constexpr int DA = BM / 32, DW = 4, LOADS = DA + DW + 2;  // direct loads a wave and block
  // Partial products in flight: tile t's second half is added in the slots of t + 2, as the
  // first instruction of t + 3 is issued.  UNROLL blocks bring every ring back to its start.
  static constexpr int PARTS = TM == 4 ? 3 : 4, UNROLL = TM == 4 ? 6 : 4;
  // Loads issued before slot I: none in the slots with most reads, two in some behind the last.
  static constexpr int loads_before(int I) {
    constexpr int wide[17] = {0, 0, 1, 2, 3, 3, 4, 5, 6, 6, 7, 8, 9, 9, 11, 13, 14};
    constexpr int narrow[9] = {0, 0, 1, 2, 3, 4, 6, 8, 10};
    return TM == 4 ? wide[I] : narrow[I < 9 ? I : 8];
  }
  // Tile rows that run together share an XCD's L2 with their columns' weights: 1024 rows (2048:
  // 4% slower over 4576 x 17408 x 5120, 8% over 16384 x 2048 x 5120; 512 and 1536: within 1%).
  static constexpr uint32_t GROUP = 1024 / BM;
  static_assert(TM == 2 || TM == 4, "schedules");
  static_assert(loads_before(2 * NT) == LOADS && NT * SLOTS % PARTS == 0 && UNROLL % SLOTS == 0 && UNROLL % 2 == 0,
                "rings");
  static_assert(LDS_BYTES <= 160 * 1024 && (SLOTS - 1) * LOADS < 64, "LDS, vmcnt range");
};

// Rows m0 .. of dx by columns k0 .., over the blocks b0 .. b0 + G - 1 of the sum (G > 0).
template <class C, bool SPLIT>
__device__ __forceinline__ void gemm_dgrad_body(const uint8_t* dy, const float* dys, const uint8_t* w,
                                                const float* ws, uint16_t* dx, float* part, uint32_t m0, uint32_t k0,
                                                uint32_t b0, uint32_t G, uint32_t split, uint32_t M, uint32_t N,
                                                uint32_t K, uint32_t Mp) {
  constexpr int TM = C::TM, TN = C::TN, SLOTS = C::SLOTS, NT = C::NT, PARTS = C::PARTS;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t wm = wave >> 1, wn = wave & 1;

  // ---- loads ----
  // The resources start at the tile; rows past M lie past dy's end and load as zeros (their
  // scales may be any of the array's values).  Every offset stays below its resource's size
  // for a row and column inside.  Wave i loads dy's rows
  // 8 DA i .. and the rows 32 i .. of w's block.
  const uint32_t blocks = N / kGroup, groups = K / kGroup, g0 = k0 / kGroup;
  const u32x4s rA = rsrc_words(dy + (uint64_t)m0 * N, (M - m0) * N);
  const u32x4s rW = rsrc_words(w + k0, N * K - k0);
  const u32x4s rAs = rsrc_words(dys + m0, (blocks * Mp - m0) * 4);
  const u32x4s rWs = rsrc_words(ws + g0, (blocks * groups - g0) * 4);
  const uint32_t l8 = lane >> 3, c8 = lane & 7;
  // (Four loads share a destination, 1 KB apart by the instruction's offset, which counts in
  // memory too: their rows are 8 apart, so what it adds can come off theirs.)
  uint32_t a_off[C::DA], w_off[C::DW], dest = 0;
#pragma unroll
  for (int j = 0; j < C::DA; ++j) a_off[j] = (8 * C::DA * wave + 8 * j + l8) * N + (c8 ^ l8 ^ (j & 1)) * 16 - j % 4 * 1024;
#pragma unroll
  for (int j = 0; j < C::DW; ++j) w_off[j] = (32 * wave + 8 * j + l8) * K + (c8 ^ l8 ^ (wave & 1)) * 16 - j % 4 * 1024;
  const uint32_t as_w = wave % TM * 256, as_off = as_w + lane * 4, ws_off = 0;
  const uint32_t lds_a = lds_addr(smem) + wave * C::DA * 1024, lds_w = lds_addr(smem) + C::W_OFF + wave * 4096;
  const uint32_t lds_as = lds_addr(smem) + C::AS_OFF + as_w, lds_ws = lds_addr(smem) + C::WS_OFF + wave * 256;
  auto load_op = [&](uint32_t b, auto slot_c, auto jc) {
    constexpr int J = decltype(jc)::value, SLOT = decltype(slot_c)::value * C::SLOT_BYTES;
    if constexpr (J < C::DA) {
      if constexpr (J % 4 == 0) dest = dma_dest<SLOT + J * 1024>(lds_a);
      dma16_to<J % 4 * 1024>(rA, a_off[J], b * kGroup, dest);
    } else if constexpr (J < C::DA + C::DW) {
      if constexpr (J == C::DA) dest = dma_dest<SLOT>(lds_w);
      dma16_to<(J - C::DA) * 1024>(rW, w_off[J - C::DA], b * kGroup * K, dest);
    } else if constexpr (J == C::DA + C::DW) {
      dma4_to(rAs, as_off, b * Mp * 4, dma_dest<SLOT>(lds_as));
    } else {
      dma4_to(rWs, ws_off, b * groups * 4, dma_dest<SLOT>(lds_ws));
    }
  };

  // ---- fragments ----
  // dy: lane l holds row l % 32, bytes 64 h + 32 (l / 32) .. of the block's half h: two chunks.
  const uint32_t l32 = lane & 31, hi = lane >> 5;
  // (Slots from the second pair on lie past what an LDS instruction's offset reaches from the
  // first; their bases are registers of their own, which the compiler must not fold together.)
  uint32_t pa[2][2][2], pw[2][TN], ps[2], pws[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      pa[0][h][c] = (wm * 32 * TM + l32) * 128 + ((4 * h + 2 * hi + c) ^ swz(l32)) * 16;
  // w: column l % 32, rows 64 h + 32 (l / 32) .., transposed
  const uint32_t row = 32 * hi + ((lane & 15) >> 1);
  const uint32_t lt = row * 128 + (swz_t(row) ^ ((lane >> 4) & 1)) * 16 + (lane & 1) * 8;
#pragma unroll
  for (int j = 0; j < TN; ++j) pw[0][j] = C::W_OFF + (lt ^ (wn * 64 + j * 32));
  ps[0] = C::AS_OFF + (wm * 32 * TM + l32) * 4;
  pws[0] = C::WS_OFF + wave * 256;
  auto upper = [](uint32_t lower) -> uint32_t {
    uint32_t u = lower + 2 * C::SLOT_BYTES;
    asm volatile("" : "+v"(u));
    return u;
  };
#pragma unroll
  for (int h = 0; h < 2; ++h) pa[1][h][0] = upper(pa[0][h][0]), pa[1][h][1] = upper(pa[0][h][1]);
#pragma unroll
  for (int j = 0; j < TN; ++j) pw[1][j] = upper(pw[0][j]);
  ps[1] = upper(ps[0]);
  pws[1] = upper(pws[0]);
  auto ld_a = [&](int sl, int i, int h, int c) -> v4i {
    return *reinterpret_cast<const v4i*>(smem + pa[sl / 2][h][c] + (sl % 2 * C::SLOT_BYTES + i * 4096));
  };
  auto ldf = [&](const uint32_t (&at)[2], int sl, int off) -> float {
    return *reinterpret_cast<const float*>(smem + at[sl / 2] + (sl % 2 * C::SLOT_BYTES + off));
  };

  v8i fy[TM - 1][2], fl[2][2], fx[2][TN][2];  // dy; its last rows and w: [set]
  float as[2][TM], wsv[2], sc[2][TM];
  v16f acc[TM][TN], p[PARTS];  // tile t of the block in slot S: p[(NT S + t) % PARTS]
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[t / TN][t % TN][r] = 0.0f;
#pragma unroll
  for (int q = 0; q < PARTS; ++q)
#pragma unroll
    for (int r = 0; r < 16; ++r) p[q][r] = 0.0f;
  sc[1][TM - 1] = 0.0f;

  // the read R of the block in slot sl into set F
  auto rd_w = [&](int sl, auto fc, auto rc) {  // 8: half of w's fragment
    constexpr int F = decltype(fc)::value, R = decltype(rc)::value, j = R / 4, h = R / 2 % 2;
    const uint8_t* at = smem + pw[sl / 2][j] + (sl % 2 * C::SLOT_BYTES + h * 8192);
    if constexpr (R & 1) fx[F][j][h].hi = ld_transposed(at, 1);
    else fx[F][j][h].lo = ld_transposed(at, 0);
  };
  auto rd_last = [&](int sl, auto fc, auto hc) {
    constexpr int F = decltype(fc)::value, h = decltype(hc)::value;
    fl[F][h].lo = ld_a(sl, TM - 1, h, 0);
    fl[F][h].hi = ld_a(sl, TM - 1, h, 1);
  };
  auto rd_a = [&](int sl, auto ic, auto hc) {
    constexpr int i = decltype(ic)::value, h = decltype(hc)::value;
    fy[i][h].lo = ld_a(sl, i, h, 0);
    fy[i][h].hi = ld_a(sl, i, h, 1);
  };
  auto rd_s = [&](int sl, auto fc, auto rc) {
    constexpr int F = decltype(fc)::value, R = decltype(rc)::value;
    as[F][2 * R] = ldf(ps, sl, R * 256);
    as[F][2 * R + 1] = ldf(ps, sl, R * 256 + 128);
  };
#define IC(n) std::integral_constant<int, (n)>{}

  // ---- prologue: three blocks of loads (past the last block the last again: in bounds,
  // never used, so that every step waits for the same count), the first into registers ----
  unroll_seq(
      [&](auto s) {
        const uint32_t b = b0 + min((uint32_t)decltype(s)::value, G - 1);
        unroll_seq([&](auto j) { load_op(b, s, j); }, std::make_integer_sequence<int, C::LOADS>{});
      },
      std::make_integer_sequence<int, SLOTS>{});
  wait_vmcnt<(SLOTS - 1) * C::LOADS>();
  wg_barrier();
  unroll_seq([&](auto r) { rd_w(0, IC(0), r); }, std::make_integer_sequence<int, 8>{});
  unroll_seq([&](auto r) { rd_a(0, IC(decltype(r)::value / 2), IC(decltype(r)::value % 2)); },
             std::make_integer_sequence<int, 2 * (TM - 1)>{});
  unroll_seq([&](auto h) { rd_last(0, IC(0), h); }, std::make_integer_sequence<int, 2>{});
  unroll_seq([&](auto r) { rd_s(0, IC(0), r); }, std::make_integer_sequence<int, TM / 2>{});
  wsv[0] = ldf(pws, 0, 0);

  // block kb, in slot S with fragments in set F
  auto step = [&](uint32_t kb, auto slot_c, auto set_c) {
    constexpr int S = decltype(slot_c)::value, F = decltype(set_c)::value;
    constexpr int nx = (S + 1) % SLOTS;
    const uint32_t lb = b0 + min(kb + SLOTS, G - 1);
    wait_lgkm0();  // this block's fragments are in registers
    sched_fence();
    unroll_seq(
        [&](auto ic) {
          constexpr int I = decltype(ic)::value, t = I / 2, h = I % 2, i = t / TN, j = t % TN;
          const v8i& a = i == TM - 1 ? fl[F][h] : fy[i < TM - 1 ? i : 0][h];
          constexpr int P = (NT * S + t) % PARTS;
          if constexpr (h == 0) {
            v16f zero;
#pragma unroll
            for (int r = 0; r < 16; ++r) zero[r] = 0.0f;
            p[P] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fx[F][j][h], a, zero, 0, 0, 0, 0, 0, 0);
          } else {
            p[P] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fx[F][j][h], a, p[P], 0, 0, 0, 0, 0, 0);
          }
          sched_fence();
          if constexpr (I == 0) {
            // the next block has landed (one block's loads are younger); every wave has read
            // this block's slot
            wait_vmcnt<(SLOTS - 2) * C::LOADS>();
            wg_barrier();
            sched_fence();
          }
          if constexpr (I == 2)
            unroll_seq([&](auto i2) { sc[F][i2] = as[F][i2] * wsv[F]; }, std::make_integer_sequence<int, TM>{});
          constexpr auto FN = IC(1 - F);
          if constexpr (TM == 4) {
            if constexpr (I == 0) rd_w(nx, FN, IC(0)), rd_w(nx, FN, IC(1));
            if constexpr (I == 1) rd_w(nx, FN, IC(2)), rd_s(nx, FN, IC(0));
            if constexpr (I == 4) rd_w(nx, FN, IC(3)), rd_w(nx, FN, IC(4));
            if constexpr (I == 5) rd_w(nx, FN, IC(5)), rd_s(nx, FN, IC(1));
            if constexpr (I == 8) rd_w(nx, FN, IC(6)), rd_w(nx, FN, IC(7));
            if constexpr (I == 9) rd_last(nx, FN, IC(0));
            if constexpr (I == 12) rd_last(nx, FN, IC(1)), wsv[1 - F] = ldf(pws, nx, 0);
          } else {
            if constexpr (I == 0) rd_w(nx, FN, IC(0)), rd_w(nx, FN, IC(1)), rd_w(nx, FN, IC(2));
            if constexpr (I == 1) rd_w(nx, FN, IC(3)), rd_w(nx, FN, IC(4)), rd_s(nx, FN, IC(0));
            if constexpr (I == 2) rd_w(nx, FN, IC(5));
            if constexpr (I == 3) rd_w(nx, FN, IC(6));
            if constexpr (I == 4) rd_w(nx, FN, IC(7)), rd_last(nx, FN, IC(0));
            if constexpr (I == 5) rd_last(nx, FN, IC(1)), wsv[1 - F] = ldf(pws, nx, 0);
          }
          if constexpr (i < TM - 1 && j == TN - 1) rd_a(nx, IC(i), IC(h));
          constexpr int L0 = C::loads_before(I), L1 = C::loads_before(I + 1);
          unroll_seq([&](auto q) { load_op(lb, slot_c, IC(L0 + decltype(q)::value)); },
                     std::make_integer_sequence<int, L1 - L0>{});
          // the first half of tile t - 1, the second of t - 2: of the block before where t is less
          constexpr int v = t - 2 + h, u = (v + NT) % NT;
          const float m = v < 0 ? sc[1 - F][u / TN] : sc[F][u / TN];
#pragma unroll
          for (int r = 8 - 8 * h; r < 16 - 8 * h; ++r) acc[u / TN][u % TN][r] += p[(NT * S + v + 2 * PARTS) % PARTS][r] * m;
          sched_fence();
        },
        std::make_integer_sequence<int, 2 * NT>{});
  };
  auto block = [&](uint32_t kb, auto sc2) {
    constexpr int I = decltype(sc2)::value;
    step(kb + I, IC(I % SLOTS), IC(I % 2));
  };
  uint32_t kb = 0;
#pragma unroll 1
  for (; kb + C::UNROLL <= G; kb += C::UNROLL)
    unroll_seq([&](auto s) { block(kb, s); }, std::make_integer_sequence<int, C::UNROLL>{});
  unroll_seq(
      [&](auto s) {
        if (kb + decltype(s)::value < G) block(kb, s);
      },
      std::make_integer_sequence<int, C::UNROLL - 1>{});
  wait_vmcnt<0>();  // no direct load may still be writing LDS when the workgroup ends
  // what the last block's last slots left
  unroll_seq(
      [&](auto s) {
        constexpr int S = decltype(s)::value % SLOTS, F = decltype(s)::value % 2;
        if ((G - 1) % C::UNROLL == decltype(s)::value) {
#pragma unroll
          for (int r = 8; r < 16; ++r) acc[TM - 1][0][r] += p[(NT * S + NT - 2) % PARTS][r] * sc[F][TM - 1];
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[TM - 1][1][r] += p[(NT * S + NT - 1) % PARTS][r] * sc[F][TM - 1];
        }
      },
      std::make_integer_sequence<int, C::UNROLL>{});
  sched_fence();

  // Lane: row 32 i + l32, columns 32 j + 8 (r / 4) + 4 (lane / 32) + r % 4.  A row group's
  // place is uniform, the lane's within it below 2^32 bytes.
  const uint32_t at = SPLIT ? l32 * K * 4 + 16 * hi : (lane & 15) * K * 2 + 32 * ((lane >> 4) & 1) + 16 * hi;
  const uint32_t mw = m0 + wm * 32 * TM;
  const uint64_t corner = (uint64_t)mw * K + k0 + wn * 64;
  const uint64_t base = SPLIT ? (uint64_t)(part + (uint64_t)split * M * K + corner) : (uint64_t)(dx + corner);
  unroll_seq(
      [&](auto ic) {
        constexpr int i = decltype(ic)::value / TN, j = decltype(ic)::value % TN;
        const v16f& c = acc[i][j];
        const uint64_t band = base + (uint64_t)(32 * i) * K * (SPLIT ? 4 : 2);
        if constexpr (SPLIT) {
          if (mw + 32 * i + l32 < M)
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
          if (mw + 32 * i + (lane & 15) < M) store16_asm<64 * j>(band, at, u32x4s{v[0][0], v[0][1], v[0][2], v[0][3]});
          if (mw + 32 * i + 16 + (lane & 15) < M)
            store16_asm<64 * j>(band + (uint64_t)16 * K * 2, at, u32x4s{v[1][0], v[1][1], v[1][2], v[1][3]});
        }
        sched_fence();
      },
      std::make_integer_sequence<int, NT>{});
#undef IC
}

}  // namespace
}  // namespace fp8q
