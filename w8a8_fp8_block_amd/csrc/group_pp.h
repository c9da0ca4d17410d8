// The ping-pong GEMM over experts' rows as one persistent pipeline: the grouped
// product's and the fused gate/up projection's kernel for many rows an expert.
#pragma once

#include "gemm_pp.h"
#include "group_tiles.h"

namespace fp8q {
namespace {

// ------------------------------------------------------------------------
// Tile 128 sorted rows x 256 columns (the ping-pong kernel's FFN layout with one
// weight matrix: group 0 computes columns 0-127, group 1 columns 128-255), so
// that an expert's last, partial row tile wastes at most 127 rows.  One
// workgroup a CU runs tiles q, q + C, q + 2C, ... as one LDS pipeline: the loads
// of the next tile follow those of the last block of the current one, so a tile
// costs no pipeline refill (with K = 2048 a tile is 16 blocks, about 14 us, and
// the refill, with the look-up of its rows, about 4).  q numbers the workgroups
// XCD by XCD, and tile ids go expert by expert (group_tile's order), so that an
// XCD's workgroups share weights and rows in its L2.
//
// The rows a tile gathers (order / per_row) are needed as load offsets when
// its first block is loaded.  They come a tile ahead, by direct loads into a
// small LDS table of two sets, so that no wave waits for them; K must hold at
// least kPersistMinBlocks blocks for them to have arrived.
//
// Bound by the matrix pipe at many rows: 36608 rows of 64 experts, N = 2048, K =
// 5120: 465 us, 1.65 PFLOP/s (1.83 with the partial tiles' rows), the pipe busy
// 43.8% of the cycles at the clock the power limit allows (the dense kernel,
// without partial tiles: 1.9-2.1, 55%); a workgroup a tile of 256 rows took 506 us
// there and 310 us for the FFN's down product (18304 rows, 32 experts, N = 5120, K =
// 2048), this kernel 260.  The fused gate/up projection of those rows (H = 5120, I =
// 2048): 515 us with a workgroup a tile, 470 us as part of the pipeline.  Near its
// lower limit of rows it is bound by the weights' stream (70 us for 288 MB at a
// mean of 51 rows: 3.1 rounds of tiles over the CUs cost the fourth round's time).
// ------------------------------------------------------------------------
constexpr uint32_t kPersistMinBlocks = 4;
constexpr uint32_t kPersistMaxExperts = 256;  // the experts' tables in LDS

struct PersistCfg {
  using C = PpCfg<3, false, true>;
  static constexpr int ROWS = C::LDS_BYTES;              // [2][128] sorted rows' order entries
  static constexpr int OFFS = ROWS + 2 * 128 * 4;        // [E + 1] first rows
  static constexpr int TILES = OFFS + (kPersistMaxExperts + 1) * 4;  // [E + 1] row tiles before
  static constexpr int RMAX = TILES + (kPersistMaxExperts + 1) * 4;  // FFN: row maxima
  static constexpr int LDS = RMAX + (int)kFfnMax;
  static_assert(LDS <= 160 * 1024, "LDS budget");
};

// WAUX: the weights' cache policy.  FFN: the experts' fused gate/up projection; W
// and Ws are gate's, ffn holds up's and the quantized intermediate [R,N], a tile's
// 256 columns are gate's and up's same 128, and out is unused.
template <int WAUX, bool FFN>
__device__ __forceinline__ void group_persist_body(const uint8_t* __restrict__ A, const float* __restrict__ As,
                                                   const uint8_t* __restrict__ W, const float* __restrict__ Ws,
                                                   uint16_t* __restrict__ out, const FfnArgs& ffn,
                                                   const Groups& g, uint32_t N, uint32_t K, uint32_t Mp,
                                                   uint32_t tiles_n) {
  using C = PersistCfg::C;
  constexpr int STAGES = 3, TM = C::TM, TN = C::TN, NP = C::NP;
  constexpr int CH0 = C::CH0, CH1 = C::CH1, LW0 = C::LW0, LW1 = C::LW1;
  constexpr uint32_t kNone = 0xFFFFFF00u;  // past any operand's bound (ceil16(rows) * K < 2^32)
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t G = K / kGroup;

  // ---- the experts' tables ----
  uint32_t* offs = reinterpret_cast<uint32_t*>(smem + PersistCfg::OFFS);
  uint32_t* tiles = reinterpret_cast<uint32_t*>(smem + PersistCfg::TILES);
  uint32_t row_tiles = 0;
  for (uint32_t b = 0; b < g.E; b += 64) {  // every wave alike
    const uint32_t e = b + lane;
    uint32_t first = 0;
    const uint32_t n = group_rows(g, e, first);
    const uint32_t scan = wave_scan_u32((n + 127) / 128, lane);
    if (wave == 0 && e < g.E) {
      offs[e] = first;
      tiles[e] = row_tiles + scan - (n + 127) / 128;
    }
    row_tiles += (uint32_t)__builtin_amdgcn_readlane((int)scan, 63);
  }
  if (threadIdx.x == 0) {
    offs[g.E] = min((uint32_t)g.offsets[g.E], g.R);
    tiles[g.E] = row_tiles;
  }
  __syncthreads();
  const uint32_t workers = gridDim.x, bid = blockIdx.x;
  const uint32_t q0 = workers % 8 == 0 ? (bid & 7) * (workers / 8) + (bid >> 3) : bid;
  const uint32_t all = row_tiles * tiles_n;
  if (q0 >= all) return;  // uniform over the workgroup

  struct Tile {
    uint32_t id, expert, m0, end, n0;
  };
  auto locate = [&](uint32_t id, Tile& t) __attribute__((always_inline)) {
    t.id = id;
    for (uint32_t b = 0;; b += 64) {
      // lane l: whether expert b + l ends after this tile
      const uint32_t e = min(b + lane, g.E - 1);
      const uint64_t past = __builtin_amdgcn_ballot_w64(tiles[e + 1] * tiles_n > id);
      if (past == 0) continue;  // (id < all: some expert holds it)
      const uint32_t x = min(b + (uint32_t)__builtin_ctzll(past), g.E - 1);
      const uint32_t before = __builtin_amdgcn_readfirstlane(tiles[x]);
      const uint32_t rt = __builtin_amdgcn_readfirstlane(tiles[x + 1]) - before;
      uint32_t tm, tn;
      grouped_tile(id - before * tiles_n, rt, tiles_n, tm, tn);
      t.expert = x;
      t.m0 = __builtin_amdgcn_readfirstlane(offs[x]) + tm * 128;
      // (an empty expert's tables repeat the next one's first row)
      t.end = __builtin_amdgcn_readfirstlane(offs[x + 1]);
      t.n0 = tn * (FFN ? 128 : 256);
      return;
    }
  };

  auto body = [&](auto grp_c) __attribute__((always_inline)) {
    constexpr uint32_t grp = decltype(grp_c)::value;
    const uint32_t gw = wave & 3;
    const uint32_t wm = gw >> 1, wn = 2 * grp + (gw & 1);
    constexpr int CH = grp ? CH1 : CH0;
    // LDS chunks (8 rows of 128 bytes): activations 0-15, columns 0-127 in
    // 16-31, 128-255 in 32-47.  Group 1 loads 16-31 and the scales of itself and
    // of its group-0 partner; group 0 activations (j < 4) and 32-47.
    auto chunk = [&](int j) __attribute__((always_inline)) -> uint32_t {
      return grp ? 16 + 4 * gw + j : j < 4 ? 4 * gw + j : 32 + 4 * gw + (j - 4);
    };
    uint32_t c_off[CH];  // weights: from the tile's first column; activations: from A
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const uint32_t row = (grp || FFN ? 4 * gw + (j & 3) : 128 / 8 + 4 * gw + (j & 3)) * 8 + (lane >> 3);
      c_off[j] = row * K + ((lane & 7) ^ swz(row)) * 16;
    }
    const uint32_t my_sc = C::A_BYTES + C::W_BYTES + wave * C::SCW_BYTES;
    const uint32_t p_sc = C::A_BYTES + C::W_BYTES + gw * C::SCW_BYTES;
    const uint32_t lds0 = lds_addr(smem);
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(A, g.a_rows * K), rS = make_rsrc(As, G * Mp * 4);
    const __amdgpu_buffer_rsrc_t rO = make_rsrc(g.order ? g.order : g.offsets, g.order ? g.R * 4 : 4);
    __amdgpu_buffer_rsrc_t rW, rWs, rWs2;  // FFN: gate's (group 1) or up's (group 0) weights; gate's, up's scales
    uint32_t s_off = 0, ws_off = 0, ws_off2 = 0;  // ws_off: columns 0-127's scales, ws_off2: 128-255's

    // ---- load cursor: tile, block, and the set of the row table it uses ----
    Tile lt;
    locate(q0, lt);
    uint32_t l_kb = 0, l_set = 0;
    bool l_more = true;
    // order entries of a tile's rows into a set of the table (wave 0's lanes
    // 0-63: rows 0-63, wave 1's: rows 64-127)
    auto fetch_rows = [&](const Tile& t, uint32_t set) __attribute__((always_inline)) {
      dma4_at(rO, g.order && t.m0 + 64 * gw + lane < t.end ? (t.m0 + 64 * gw + lane) * 4 : kNone, 0,
              lds0 + PersistCfg::ROWS + set * 512 + 256 * gw);
    };
    // this wave's load offsets for the tile lt, whose rows are in set l_set
    auto offsets_of = [&]() __attribute__((always_inline)) {
      const uint32_t* rows = reinterpret_cast<const uint32_t*>(smem + PersistCfg::ROWS) + l_set * 128;
      auto src = [&](uint32_t r) __attribute__((always_inline)) -> uint32_t {  // activation row of tile row r
        const uint32_t m = g.order ? rows[r] / g.per_row : lt.m0 + r;
        return min(m, g.a_rows - 1);
      };
      if constexpr (grp == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t r = (4 * gw + j) * 8 + (lane >> 3);
          c_off[j] = lt.m0 + r < lt.end ? src(r) * K + ((lane & 7) ^ swz(r)) * 16 : kNone;
        }
      } else {
        const uint32_t r = wm * C::WM + lane;
        s_off = src(min(r, lt.end - 1 - lt.m0)) * 4;
        ws_off = scale_row(lt.n0, 0, N) * G * 4;
        ws_off2 = scale_row(lt.n0, 1, N) * G * 4;
        rWs = make_rsrc(Ws + (uint64_t)lt.expert * (N / kGroup) * G, (N / kGroup) * G * 4);
        if constexpr (FFN) rWs2 = make_rsrc(ffn.ws_up + (uint64_t)lt.expert * (N / kGroup) * G, (N / kGroup) * G * 4);
      }
      // columns past N (N / 128 odd): out of range, zeros
      rW = make_rsrc((FFN && grp == 0 ? ffn.w_up : W) + ((uint64_t)lt.expert * N + lt.n0) * K, (N - lt.n0) * K);
    };
    // the next block, or the first of the next tile
    Tile nt;  // the tile after lt
    auto load_next = [&]() __attribute__((always_inline)) {
      if (++l_kb < G) return;
      if (!l_more) {  // past the last tile: its last block again (never read)
        l_kb = G - 1;
        return;
      }
      l_kb = 0;
      lt = nt;
      l_set ^= 1;
      offsets_of();
      l_more = lt.id + workers < all;
      if (l_more) locate(lt.id + workers, nt);
    };
    auto issue = [&](uint32_t stage) __attribute__((always_inline)) {
      uint32_t lds = lds0 + stage * C::STAGE_BYTES;
      asm volatile("" : "+s"(lds));
      const uint32_t kb = l_kb;
      unroll_seq(
          [&](auto jc) {
            constexpr int J = decltype(jc)::value;
            if constexpr (grp == 0 && J < 4)
              dma16_at(rA, c_off[J], kb * kGroup, lds + chunk(J) * 1024);
            else
              dma16_at_aux<WAUX>(rW, c_off[J], kb * kGroup, lds + chunk(J) * 1024);
          },
          std::make_integer_sequence<int, CH>{});
      if constexpr (grp == 1) {
        dma4_at(rS, s_off, kb * Mp * 4, lds + my_sc);
        dma4_at(rS, s_off, kb * Mp * 4, lds + p_sc);  // (the partner: the same rows)
        if constexpr (FFN)
          dma4_at(rWs2, 0, ws_off + kb * 4, lds + my_sc + 256);
        else
          dma4_at(rWs, 0, ws_off2 + kb * 4, lds + my_sc + 256);
        dma4_at(rWs, 0, ws_off + kb * 4, lds + p_sc + 256);
      }
      // with a tile's first block: the row table of the tile after it (waves 0
      // and 1 of group 0; the set it overwrites was last read a tile ago)
      if (grp == 0 && gw < 2 && kb == 0 && l_more) fetch_rows(nt, l_set ^ 1);
      load_next();
    };

    const uint32_t l16 = lane & 15, c0 = 2 * (lane >> 4);
    const uint32_t lo0 = l16 * 128 + ((c0 ^ swz(l16)) * 16);
    const uint32_t lo1 = l16 * 128 + (((c0 + 1) ^ swz(l16)) * 16);
    auto ld16 = [](const uint8_t* p) __attribute__((always_inline)) -> v4i { return *reinterpret_cast<const v4i*>(p); };
    auto ldf = [](const uint8_t* p) __attribute__((always_inline)) -> float { return *reinterpret_cast<const float*>(p); };
    const uint32_t a_row0 = wm * C::WM * 128, w_row0 = C::A_BYTES + wn * C::WN * 128;

    v4f acc[TM][TN];
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    };
    clear();
    v8i af[TM], bf[TN];
    float as[TM], ws = 0.0f, sc[TM], sc_tail = 0.0f;
    v4f p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    auto read_block = [&](auto slot_c) __attribute__((always_inline)) {
      const uint8_t* sb = smem + decltype(slot_c)::value * C::STAGE_BYTES;
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        bf[tn].lo = ld16(sb + w_row0 + tn * 2048 + lo0);
        bf[tn].hi = ld16(sb + w_row0 + tn * 2048 + lo1);
      }
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        af[tm].lo = ld16(sb + a_row0 + tm * 2048 + lo0);
        af[tm].hi = ld16(sb + a_row0 + tm * 2048 + lo1);
        as[tm] = ldf(sb + my_sc + (tm * 16 + l16) * 4);
      }
      ws = ldf(sb + my_sc + 256);
    };
    auto compute_block = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) sc[tm] = as[tm] * ws;
      unroll_seq(
          [&](auto ic) {
            constexpr int I = decltype(ic)::value;
            constexpr int tm = I / TN, tn = I % TN;
            p[I & 3] = mfma_e4m3_128(bf[tn], af[tm]);
            // each promotion pinned to its slot (see the stream-K kernel)
            if constexpr (I < kPromoteDist) {
              constexpr int J = NP - kPromoteDist + I;
              acc[J / TN][J % TN] += p[J & 3] * sc_tail;
              asm volatile("" : "+v"(acc[J / TN][J % TN]));
            } else {
              constexpr int J = I - kPromoteDist;
              acc[J / TN][J % TN] += p[J & 3] * sc[J / TN];
              asm volatile("" : "+v"(acc[J / TN][J % TN]));
            }
            sched_fence();
          },
          std::make_integer_sequence<int, NP>{});
      sc_tail = sc[TM - 1];
    };
    Tile ct = lt;  // compute cursor
    auto promote_rest = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int j = NP - kPromoteDist; j < NP; ++j) acc[j / TN][j % TN] += p[j & 3] * sc_tail;
      sc_tail = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    };
    auto epilogue = [&]() __attribute__((always_inline)) {
      promote_rest();
      if (ct.n0 + wn * C::WN < N) {
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
          const uint32_t m = ct.m0 + wm * C::WM + tm * 16 + l16;
          if (m < ct.end) {
#pragma unroll
            for (int tn = 0; tn < TN; ++tn) {
              const uint32_t n = ct.n0 + wn * C::WN + tn * 16 + 4 * (lane >> 4);
              *reinterpret_cast<uint2*>(out + (uint64_t)m * N + n) = pack_bf16x4(acc[tm][tn]);
            }
          }
        }
      }
      clear();
    };

    auto half0 = [&](auto slot_c) __attribute__((always_inline)) {
      constexpr int S = decltype(slot_c)::value;
      if constexpr (grp == 0) {
        compute_block();
        wait_vmcnt<LW0>();
        wg_barrier();
      } else {
        read_block(slot_c);
        wait_lgkm0();
        issue(S);
        wait_vmcnt<2 * LW1>();
        wg_barrier();
      }
    };
    auto half1 = [&](auto slot_c) __attribute__((always_inline)) {
      constexpr int S = decltype(slot_c)::value;
      if constexpr (grp == 0) {
        read_block(std::integral_constant<int, (S + 1) % STAGES>{});
        wait_lgkm0();
        issue(S);
        wg_barrier();
      } else {
        compute_block();
        wg_barrier();
      }
    };
    auto step = [&](auto slot_c) __attribute__((always_inline)) {
      half0(slot_c);
      half1(slot_c);
    };
    auto dispatch = [&](uint32_t sl, auto&& half) __attribute__((always_inline)) {
      if (sl == 0)
        half(std::integral_constant<int, 0>{});
      else if (sl == 1)
        half(std::integral_constant<int, 1>{});
      else
        half(std::integral_constant<int, 2>{});
    };
    // FFN: a tile's last block, in slot sl, with its epilogue.  The slot's refill
    // waits until the epilogue has used it: both groups have read the block
    // after half 0, the waves exchange gate and up through it, and after the
    // second exchange barrier it is free again.  At the next block's waits as many
    // loads are in flight as without (and this tile's stores, which are older).
    auto last_ffn = [&](uint32_t sl) __attribute__((always_inline)) {
      uint8_t* slot = smem + sl * C::STAGE_BYTES;
      uint16_t* rmax = reinterpret_cast<uint16_t*>(smem + PersistCfg::RMAX);
      if constexpr (grp == 0) {
        compute_block();
        wait_vmcnt<LW0>();
        wg_barrier();
      } else {
        dispatch(sl, read_block);
        wait_lgkm0();
        wait_vmcnt<LW1>();  // own part of the next block
        wg_barrier();
        compute_block();
      }
      promote_rest();
      ffn_park<TM, TN>(acc, slot, wave, lane);
      wait_lgkm0();
      wg_barrier();
      uint32_t hb[2][TN][2], amax[2];
      ffn_h<TM, TN>(acc, slot, rmax, wave, lane, hb, amax);
      wait_lgkm0();
      wg_barrier();
      ffn_codes<TN>(hb, amax, rmax, ffn, wave, lane, ct.m0 + wm * C::WM, ct.n0 + (gw & 1) * C::WN, ct.n0 / kGroup,
                    ct.end, N, ct.end);
      issue(sl);
      if constexpr (grp == 0) {
        dispatch(sl == 2 ? 0 : sl + 1, read_block);
        wait_lgkm0();
      }
      wg_barrier();
      clear();
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    using S2 = std::integral_constant<int, 2>;

    // the first tile's rows (needed at once), then the pipeline's first loads
    if (grp == 0 && gw < 2) {
      fetch_rows(lt, 0);
      wait_vmcnt<0>();
    }
    wg_barrier();
    offsets_of();
    l_more = lt.id + workers < all;
    if (l_more) locate(lt.id + workers, nt);
#pragma unroll
    for (int st = 0; st < STAGES; ++st) issue(st);
    if constexpr (grp == 0) {
      wait_vmcnt<(STAGES - 1) * LW0>();
      wg_barrier();
      read_block(S0{});
      wait_lgkm0();
      wg_barrier();
    } else {
      wait_vmcnt<(STAGES - 1) * LW1>();
      wg_barrier();
      wg_barrier();
    }
    // blocks i counted over the workgroup's tiles (slot i % 3); a tile's last
    // block with its epilogue, where the group holds nothing but accumulators
    uint32_t i = 0;
    while (true) {
      const uint32_t last = i + G - 1;
      const uint32_t ph = i % 3;
      if (ph == 1 && i < last) {
        step(S1{});
        ++i;
      }
      if (i % 3 == 2 && i < last) {
        step(S2{});
        ++i;
      }
      for (; i + 3 <= last; i += 3) {
        step(S0{});
        step(S1{});
        step(S2{});
      }
      if (i < last) {
        step(S0{});
        ++i;
      }
      if (i < last) {
        step(S1{});
        ++i;
      }
      if constexpr (FFN) {
        last_ffn(i % 3);
      } else {
        dispatch(i % 3, half0);
        if constexpr (grp == 0) epilogue();
        dispatch(i % 3, half1);
        if constexpr (grp == 1) epilogue();
      }
      ++i;
      if (ct.id + workers >= all) break;
      locate(ct.id + workers, ct);
    }
    wait_vmcnt<0>();  // no direct load may still be writing LDS at exit
  };
  if (wave >> 2)
    body(std::integral_constant<uint32_t, 1>{});
  else
    body(std::integral_constant<uint32_t, 0>{});
}

template <int WAUX>
__global__ __launch_bounds__(512) void group_persist_kernel(const uint8_t* __restrict__ A,
                                                            const float* __restrict__ As,
                                                            const uint8_t* __restrict__ W,
                                                            const float* __restrict__ Ws,
                                                            uint16_t* __restrict__ out, Groups g, uint32_t N,
                                                            uint32_t K, uint32_t Mp, uint32_t tiles_n) {
  group_persist_body<WAUX, false>(A, As, W, Ws, out, FfnArgs{nullptr, nullptr, nullptr, nullptr, 0}, g, N, K, Mp,
                                  tiles_n);
}

template <int WAUX>
__global__ __launch_bounds__(512) void group_persist_ffn_kernel(const uint8_t* __restrict__ A,
                                                                const float* __restrict__ As,
                                                                const uint8_t* __restrict__ w_gate,
                                                                const float* __restrict__ ws_gate, FfnArgs ffn,
                                                                Groups g, uint32_t I, uint32_t H, uint32_t Mp,
                                                                uint32_t tiles_n) {
  group_persist_body<WAUX, true>(A, As, w_gate, ws_gate, nullptr, ffn, g, I, H, Mp, tiles_n);
}

}  // namespace
}  // namespace fp8q
