// What a GEMM tile's output rows are: the policies of the kernel bodies.
//
//   total             activation rows (the operand's bound)
//   end               first row past the tile's rows: rows from here on are
//                     neither stored nor counted
//   src(m)            activation row that output row m < end reads
//   scale_slot(m, Mp) its slot in the K-major scales (any m; in bounds)
//   pad_end(Mp)       K-major output scales of rows end .. pad_end-1 are
//                     written zero (the FFN epilogue's pad slots)
#pragma once

#include "mfma_common.h"

namespace fp8q {
namespace {

// Output row m reads activation row m.
struct DenseRows {
  uint32_t total, end;
  __device__ __forceinline__ uint32_t src(uint32_t m) const { return m; }
  __device__ __forceinline__ uint32_t scale_slot(uint32_t m, uint32_t Mp) const { return min(m, Mp - 1); }
  __device__ __forceinline__ uint32_t pad_end(uint32_t Mp) const { return Mp; }
};

// Adds nothing to the accumulators.  An epilogue adds to a wave's TM x TN tiles of
// 16 x 16, called by the whole workgroup with its LDS: `add` in the tiled kernels,
// where the wave's rows are band.. of the workgroup's BM, `add_shared` in the
// decode-width ones, where the waves hold the same rows and columns.
struct NoEpilogue {
  template <int TM, int TN, int NT, int BM, class Acc>
  __device__ __forceinline__ void add(Acc&&, uint8_t*, uint32_t, uint32_t, uint32_t, uint32_t, uint32_t,
                                      uint32_t) const {}
  template <int TM, int TN, int NT, class Acc>
  __device__ __forceinline__ void add_shared(Acc&&, uint8_t*, uint32_t, uint32_t, uint32_t, uint32_t, uint32_t,
                                             uint32_t) const {}
};

}  // namespace
}  // namespace fp8q
