// The decode-width GEMM kernels (skinny and decode), their register and grid
// rules and kernel bodies, shared by the dense kernels (gemm.hip) and the
// projection with per-request adapters (lora.hip).
#pragma once

#include <algorithm>

#include "gemm_tile.h"

namespace fp8q {
namespace {

// ------------------------------------------------------------------------
// Skinny kernel for decode and small-batch widths.  Rows come in tiles of
// 16*TM <= 64 (grid dimension y; beyond 64 rows every row tile streams the
// weights again, mostly from the last-level cache).  The projection is then
// bound by streaming the weight matrix once, and the weight bytes must be
// spread evenly over the CUs: with one workgroup per 16 output columns
// (384 workgroups at N = 6144 on 256 CUs) half the CUs stream twice as much
// as the others.  So the grid has one workgroup per CU and workgroup w owns
// the contiguous column range [c0, c0 + cw), cw = N/grid rounded to 4
// columns, covered by ceil(cw/16) MFMA tiles of 16 columns (the last one
// partial: its missing weight rows are zero fragments, its missing columns
// are not stored).  The NWV waves take interleaved K blocks (wave w: blocks
// w, w+NWV, ...) for all of the workgroup's tiles; each wave issues the loads
// of U blocks before consuming any, the activation fragments of a block are
// loaded once for all tiles, and the NWV partial tiles are summed through
// LDS in wave order.
// ------------------------------------------------------------------------
// SPLIT: the K blocks are cut into gridDim.z contiguous ranges; workgroup
// (w, y, z) sums range z and stores its fp32 partial tile to part[z][M][N],
// which splitk_reduce_kernel adds in split order (block-scaled weights only).
// Epi adds to the waves' partial sums before they are joined, its work dealt
// over the waves (and splits).
template <int TM, int TN, int NWV, int U, bool ROW, bool SPLIT, class Epi>
__device__ __forceinline__ void gemm_skinny_body(
    const uint8_t* __restrict__ A, const float* __restrict__ As, const uint8_t* __restrict__ W,
    const float* __restrict__ Ws, uint16_t* __restrict__ out, uint32_t M, uint32_t N, uint32_t K,
    uint32_t Mp, uint32_t units_base, uint32_t units_rem, float* __restrict__ part, const Epi& epi) {
#include "gemm_skinny_body.h"
}

// ------------------------------------------------------------------------
// Decode-width kernel for the shapes whose per-workgroup weight slice fits
// in LDS (up to 32 rows, 16*TM <= 32 activation rows, at most 8*GW K
// blocks).  The projection streams the weight matrix once from HBM, and how
// the weight bytes are read decides its speed: fragment-layout loads (lane
// l: 32 bytes of row l%16, gemm_skinny_kernel) touch 16 rows K bytes apart
// with every instruction, while direct-to-LDS loads of whole 1 KB row pieces,
// all in flight at once, stream the same bytes about 1.6x faster (N = 6144,
// K = 5120 on 256 CUs, the weight read alone from HBM: 6.8 us against 10.7
// us).  Workgroup w owns the contiguous column range [c0, c0 + R) as in
// gemm_skinny_kernel; it loads the R weight rows into LDS (each row's K bytes
// contiguous and followed by a 16-byte pad, so that the 16 rows of an MFMA
// fragment read fall in 16 different bank quads), and, into registers, the
// activation fragments and the scales of the K blocks its waves take (wave
// v: blocks v, v+8, ..., every row tile, as gemm_skinny_kernel), all before
// the first wait.  Then the waves compute their blocks and add the 8 partial
// tiles in wave order through LDS: the same products as gemm_skinny_kernel,
// each wave's blocks added in an order rotated by the workgroup index.
// Measured at N = 6144, K = 5120 (weights from HBM, graph-timed back-to-back
// launches): 9.5 / 11.0 / 11.7 us at M = 16 / 17 / 25 against 12.6 / 14.0 /
// 14.8 us for gemm_skinny_kernel.  What remains above the bare weight stream
// is the activation reads (every workgroup reads all M x K activation bytes
// through its vector memory unit ahead of its weight loads: 0.7 us at M = 16,
// 2 us at M = 25) and the products, the reduction and the store after the
// single wait (about 1.8 us).  Waiting for the weight loads stage by stage,
// one K slot at a time, was slower: the barriers cost more than the overlap
// gains.
// ------------------------------------------------------------------------
constexpr uint32_t kDecodeMaxRows = 32, kDecodeLds = 150 * 1024;

template <int TM, int GW, bool ROW, class Epi>
__device__ __forceinline__ void gemm_decode_body(
    const uint8_t* __restrict__ A, const float* __restrict__ As, const uint8_t* __restrict__ W,
    const float* __restrict__ Ws, uint16_t* __restrict__ out, uint32_t M, uint32_t N, uint32_t K,
    uint32_t Mp, uint32_t units_base, uint32_t units_rem, const Epi& epi) {
#include "gemm_decode_body.h"
}

// Whether the decode kernel takes the shape (its limits: at most 32 rows and
// kDecodeMaxRows columns a workgroup, 48 K blocks, the slice within
// kDecodeLds), and then its template arguments and LDS bytes.
bool decode_plan(uint32_t M, uint32_t K, uint32_t base, uint32_t rem, uint32_t& tm, uint32_t& gw,
                 uint32_t& lds) {
  const uint32_t rmax = 4 * (base + (rem ? 1 : 0)), g = (K / kGroup + 7) / 8;
  const uint64_t l = std::max<uint64_t>((uint64_t)rmax * (K + 16), 8 * 2 * 2 * 64 * 16);
  if (M > 32 || rmax > kDecodeMaxRows || g > 6 || l > kDecodeLds) return false;
  tm = M <= 16 ? 1 : 2;
  gw = g <= 2 ? 2 : g <= 4 ? 4 : g == 5 ? 5 : 6;
  lds = (uint32_t)l;
  return true;
}

// Registers of a skinny wave: about 4*TN*TM accumulators + 4*TN + 3*TM + 20
// fixed, 9*TN + 9*TM per K block in flight.
constexpr int skinny_fixed_regs(int tm, int tn) { return 4 * tn * tm + 4 * tn + 3 * tm + 20; }
constexpr int skinny_block_regs(int tm, int tn) { return 9 * tn + 9 * tm; }
// Two waves per SIMD wherever the partial sums of eight fit in 128 KB of LDS,
// with the K blocks in flight that ~242 registers a wave leave (at least
// one).  Measured against one wave per SIMD with more blocks in flight (cold
// caches): TM = 2, TN = 6 (17-32 rows, N = 17408, K = 5120; two blocks
// against four): 28.9 / 30.1 / 30.8 against 31.4 / 32.5 / 33.2 us at M = 17
// / 25 / 32; TM = 4, TN = 4 (65-128 rows in 64-row tiles, 64 columns a
// workgroup; one block against four): 78.4-80.3 against 87.1-90.0 us at
// N = 5120, K = 17408 and 28.4-30.5 against 32.0-34.2 at N = 6144, K = 5120.
constexpr bool skinny_two_per_simd(int tm, int tn) { return 8 * tn * tm <= 128; }
// waves per workgroup: 8 where the rule above holds, else 4 where the
// partial sums of 4 fit in 128 KB (one wave per SIMD), else 2
constexpr int skinny_waves(int tm, int tn) {
  return skinny_two_per_simd(tm, tn) ? 8 : (128 / (tn * tm) >= 4) ? 4 : 2;
}
// K blocks in flight per wave: what the register budget leaves (~200 a wave
// at two waves per SIMD where eight waves' partial sums fit in 64 KB, as
// first tuned; 242 for the wider configurations; ~440 at one wave per SIMD)
constexpr int skinny_unroll(int tm, int tn) {
  const int budget = skinny_waves(tm, tn) != 8 ? 440 : (64 / (tn * tm) >= 8) ? 200 : 242;
  const int uf = (budget - skinny_fixed_regs(tm, tn)) / skinny_block_regs(tm, tn);
  return uf > 8 ? 8 : uf < 1 ? 1 : uf;
}
// the template arguments the skinny dispatch picks: row tiles TM of 16 rows,
// column tiles TN of 16 columns.  TM = 3 for 33-48 rows: against TM = 4 it
// leaves the registers for two K blocks in flight at TN = 4 (one at TM =
// 4) and loads a quarter fewer activation fragments; back to back over
// rotating weights, M = 33 / 48: single pass 41.1 / 46.4 -> 36.7 / 42.9 us
// at N = 5120, K = 17408 (3 splits 33.0 / 35.0 -> 30.3 / 32.8), 34.6 / 35.9
// -> 31.8 / 33.4 at N = 17408, K = 5120, 16.3 / 17.8 -> 15.2 / 16.9 at
// N = 6144, K = 5120.
uint32_t skinny_tm(uint32_t M) { return M <= 16 ? 1 : M <= 32 ? 2 : M <= 48 ? 3 : 4; }
uint32_t skinny_tn(uint32_t tn) { return tn <= 2 ? 2 : tn <= 4 ? 4 : tn <= 6 ? 6 : 8; }

// The skinny path's grid.  Up to 64 rows (one row tile): one workgroup per
// CU, at most 128 columns each, at least 16.  Beyond (several row tiles,
// each streaming the weights again): workgroups of 64 columns, so that a row
// tile re-reads the activations once per 64 columns rather than once per CU
// (measured at M = 128, N = 5120, K = 17408: 90 us with 64-column
// workgroups, 108 us with one per CU, 117 us for the ping-pong kernel).
// Workgroup w owns 4*(base + (w < rem)) columns; tn 16-column tiles at most.
void skinny_grid(uint32_t M, uint32_t N, uint32_t cu_count, uint32_t& grid, uint32_t& base,
                 uint32_t& rem, uint32_t& tn) {
  const uint32_t units = N / 4;
  grid = max(cu_count, (N + 127) / 128);
  grid = max(1u, min(grid, N / 16));
  if (M > 64) grid = N / 64;
  base = units / grid;
  rem = units % grid;
  tn = (4 * (base + (rem ? 1 : 0)) + 15) / 16;
}

}  // namespace
}  // namespace fp8q
