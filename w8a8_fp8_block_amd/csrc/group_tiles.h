// Tiles of products grouped by expert: rows sorted by expert, group e at rows
// offsets[e] .. offsets[e + 1], known on the device only.  A launch's grid
// covers the most tiles any distribution of the rows can have; each workgroup
// finds its tile from the offsets, and those past the last tile end at once.
#pragma once

#include "mfma_common.h"

namespace fp8q {
namespace {

struct Groups {
  const int32_t* offsets;  // [E + 1]
  const int32_t* order;    // sorted row -> slot; NULL: output row p reads activation row p
  uint32_t E, R;           // groups; sorted rows
  uint32_t per_row;        // slots per activation row: sorted row p reads row order[p] / per_row
  uint32_t a_rows;         // activation rows
};

// Rows of one expert: output row p (a sorted row) reads activation row
// order[p] / per_row.  Everything is clamped in bounds, whatever the plan holds.
struct GroupRows {
  uint32_t total, end;
  const int32_t* order;
  uint32_t per_row;
  __device__ __forceinline__ uint32_t src(uint32_t m) const {
    return min(order ? (uint32_t)order[m] / per_row : m, total - 1);
  }
  __device__ __forceinline__ uint32_t scale_slot(uint32_t m, uint32_t) const { return src(min(m, end - 1)); }
  __device__ __forceinline__ uint32_t pad_end(uint32_t) const { return end; }
};

struct GroupTile {
  uint32_t expert, m0, end, tn;  // first row, end of the expert's rows, column tile
};

// inclusive sum over the wave's lanes up to this one
__device__ __forceinline__ uint32_t wave_scan_u32(uint32_t v, uint32_t lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)v, d);
    if (lane >= (uint32_t)d) v += o;
  }
  return v;
}

// rows of expert e, the first of them in `first`
__device__ __forceinline__ uint32_t group_rows(const Groups& g, uint32_t e, uint32_t& first) {
  if (e >= g.E) return 0;
  first = min((uint32_t)g.offsets[e], g.R);
  const uint32_t last = min((uint32_t)g.offsets[e + 1], g.R);
  return last > first ? last - first : 0;
}

// The row tiles of BM rows, expert by expert, seen by a wave: lane l holds
// expert l's rows (and, beyond 64 experts, looks the later ones up again).
template <uint32_t BM>
struct RowTiles {
  uint32_t lane, n = 0, first = 0, scan = 0;  // expert `lane`: rows, first row, row tiles up to it
  uint32_t total;                             // row tiles in all

  __device__ __forceinline__ RowTiles(const Groups& g, uint32_t lane_) : lane(lane_) {
    n = group_rows(g, lane, first);
    scan = wave_scan_u32((n + BM - 1) / BM, lane);
    total = (uint32_t)__builtin_amdgcn_readlane((int)scan, 63);
    for (uint32_t b = 64; b < g.E; b += 64) {
      uint32_t f;
      const uint32_t s = wave_scan_u32((group_rows(g, b + lane, f) + BM - 1) / BM, lane);
      total += (uint32_t)__builtin_amdgcn_readlane((int)s, 63);
    }
  }

  // The expert whose run of tiles (each row tile counting `each`) holds tile
  // id < total * each: expert, its first row, end, and the tiles before it.
  __device__ __forceinline__ void find(const Groups& g, uint32_t id, uint32_t each, uint32_t& expert,
                                       uint32_t& row0, uint32_t& end, uint32_t& prior) {
    uint32_t before = 0;
    for (uint32_t b = 0;; b += 64) {
      if (b) {
        n = group_rows(g, b + lane, first);
        scan = wave_scan_u32((n + BM - 1) / BM, lane);
      }
      const uint64_t past = __builtin_amdgcn_ballot_w64((before + scan) * each > id);
      if (past) {
        const int l = __builtin_ctzll(past);
        const uint32_t rows = (uint32_t)__builtin_amdgcn_readlane((int)n, l);
        expert = b + (uint32_t)l;
        row0 = (uint32_t)__builtin_amdgcn_readlane((int)first, l);
        end = row0 + rows;
        prior = (before + (uint32_t)__builtin_amdgcn_readlane((int)scan, l) - (rows + BM - 1) / BM) * each;
        return;
      }
      before += (uint32_t)__builtin_amdgcn_readlane((int)scan, 63);
    }
  }
};

// This workgroup's tile of BM rows (false: none left).  Tile ids go expert by
// expert; within one, blocks of up to 8 row tiles with the column tiles outside,
// so that neighbours share weight columns, then activation rows; each XCD takes
// a contiguous run of ids (workgroup ids are dealt round robin to the 8 XCDs).
template <uint32_t BM>
__device__ __forceinline__ bool group_tile(const Groups& g, uint32_t tiles_n, uint32_t bid,
                                           uint32_t lane, GroupTile& t) {
  RowTiles<BM> rt(g, lane);
  const uint32_t total = rt.total * tiles_n, xcd = bid & 7, slot = bid >> 3;
  const uint32_t q = total >> 3, r8 = total & 7;
  if (slot >= q + (xcd < r8 ? 1 : 0)) return false;
  const uint32_t id = xcd * q + min(xcd, r8) + slot;
  uint32_t row0, prior, tm;
  rt.find(g, id, tiles_n, t.expert, row0, t.end, prior);
  grouped_tile(id - prior, (t.end - row0 + BM - 1) / BM, tiles_n, tm, t.tn);
  t.m0 = row0 + tm * BM;
  return true;
}

// Weight-scale row (of N / 128) of columns n0 + 128 * half .. + 127.  A 256-column
// tile's second half may lie past N (N / 128 odd): its results are not stored, and it
// takes the last row, since a scale's place is a load's scalar offset, which the
// buffer's bound does not hold.
__host__ __device__ __forceinline__ uint32_t scale_row(uint32_t n0, uint32_t half, uint32_t N) {
  const uint32_t row = n0 / kGroup + half, last = N / kGroup - 1;
  return row < last ? row : last;
}

// Most row tiles of bm rows that R rows in E groups can need.
inline uint32_t max_row_tiles(uint32_t R, uint32_t E, uint32_t bm) {
  const uint64_t g = R < E ? R : E;
  return (uint32_t)((R + g * (bm - 1)) / bm);
}

}  // namespace
}  // namespace fp8q
