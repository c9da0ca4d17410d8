// What the two gradient products (gemm_dgrad.h, gemm_wgrad.h) share: direct loads issued in
// assembly, LDS reads that transpose, and stores of 32 x 32 tiles of accumulators.
#pragma once

#include "mfma_common.h"

namespace fp8q {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

// A buffer resource's words.  Lanes copy 16 or 4 bytes each from its base + voff + soff +
// OFF to lds + LDS_OFF onwards (the instruction adds its offset on both sides; M0 holds no
// other value in these kernels).  In assembly because the compiler takes ld_transposed's
// read for one of any LDS in flight and would wait for every direct load it knows of before
// it; these it does not know, and every wait is the kernel's own.
typedef uint32_t u32x4s __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4s rsrc_words(const void* base, uint32_t bytes) {
  const uint64_t p = (uint64_t)base;
  return u32x4s{(uint32_t)p, (uint32_t)(p >> 32) & 0xFFFFu, bytes, 0x00020000u};
}
template <int OFF, int LDS_OFF>
__device__ __forceinline__ void dma16_asm(u32x4s r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_add_u32 m0, %3, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen offset:%5 lds"
               :: "v"(voff), "s"(r), "s"(soff), "s"(lds), "n"(LDS_OFF - OFF), "n"(OFF) : "memory", "scc");
}
template <int LDS_OFF>
__device__ __forceinline__ void dma4_asm(u32x4s r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_add_u32 m0, %3, %4\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
               :: "v"(voff), "s"(r), "s"(soff), "s"(lds), "n"(LDS_OFF) : "memory", "scc");
}

// The same with the destination set apart from the loads, for several loads to one: lds + OFF.
template <int OFF>
__device__ __forceinline__ uint32_t dma_dest(uint32_t lds) {
  uint32_t m0;
  asm volatile("s_add_u32 %0, %1, %2\n\ts_nop 0" : "={m0}"(m0) : "s"(lds), "n"(OFF) : "scc");
  return m0;
}
template <int OFF>
__device__ __forceinline__ void dma16_to(u32x4s r, uint32_t voff, uint32_t soff, uint32_t dest) {
  asm volatile("buffer_load_dwordx4 %0, %1, %2 offen offset:%3 lds"
               :: "v"(voff), "s"(r), "s"(soff), "n"(OFF), "{m0}"(dest) : "memory");
}
__device__ __forceinline__ void dma4_to(u32x4s r, uint32_t voff, uint32_t soff, uint32_t dest) {
  asm volatile("buffer_load_dword %0, %1, %2 offen lds" :: "v"(voff), "s"(r), "s"(soff), "{m0}"(dest) : "memory");
}

// A matrix whose rows are the sum's index: a panel of rows of 128 bytes (columns), 16-byte
// chunk c of row r at chunk position c ^ swz_t(r).  ds_read_b64_tr_b8 takes 8 bytes from
// each lane of a 16-lane row and gives lane l byte l % 8 of the lanes 2j + l / 8, j = 0..7:
// with lane 2j + h at row j, bytes 8h.. of a chunk, lane l gets column l of the chunk's 16
// in 8 rows.  Four of them, 8 rows apart, fill the 32 rows that a lane holds of a fragment,
// in order.  swz_t spreads the 8 rows of a 16-lane row over the 8 chunk positions, and those
// of the lanes that are read together over chunks of different parity.
__device__ __forceinline__ uint32_t swz_t(uint32_t r) { return (r & 7u) ^ ((r >> 5) & 1u); }
typedef int v2i __attribute__((ext_vector_type(2)));

// half h (16 rows) of the fragment whose lane's place p is
__device__ __forceinline__ v4i ld_transposed(const uint8_t* p, int h) {
  typedef __attribute__((address_space(3))) v2i lds_v2i;
  const v2i a = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)(p + h * 2048));
  const v2i b = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)(p + h * 2048 + 1024));
  return v4i{a.x, a.y, b.x, b.y};
}

// 16 bytes a lane to base + voff + OFF.  (In assembly for the uniform base: with an address
// a lane, the tile's end spills, and each reload waits for the stores.  The data's
// registers may be written two instructions later.)
template <int OFF>
__device__ __forceinline__ void store16_asm(uint64_t base, uint32_t voff, u32x4s v) {
  asm volatile("global_store_dwordx4 %0, %1, %2 offset:%3\n\ts_nop 1" ::"v"(voff), "v"(v), "s"(base), "n"(OFF)
               : "memory");
}

// A 32 x 32 tile's accumulators as bf16 for two stores of 16 rows x 64 bytes, not 32 x 32:
// v[s] is row 16 s + lane % 16, 16 bytes at 32 (lane / 16 % 2) + 16 (lane / 32).  Lane l
// holds four columns in four of each row's eight places; the halves of the wave swap (8
// columns a lane), then the odd and even 16-lane rows.
__device__ __forceinline__ void tile_rows_bf16(const v16f& c, uint32_t (&v)[2][4]) {
  unroll_seq(
      [&](auto rc) {
        constexpr int s = decltype(rc)::value, r = 8 * s;
        const auto s0 = __builtin_amdgcn_permlane32_swap(bf16x2_rne(c[r], c[r + 1]),
                                                         bf16x2_rne(c[r + 4], c[r + 5]), false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(bf16x2_rne(c[r + 2], c[r + 3]),
                                                         bf16x2_rne(c[r + 6], c[r + 7]), false, false);
        v[s][0] = s0[0], v[s][1] = s1[0], v[s][2] = s0[1], v[s][3] = s1[1];
      },
      std::make_integer_sequence<int, 2>{});
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const auto s = __builtin_amdgcn_permlane16_swap(v[0][d], v[1][d], false, false);
    v[0][d] = s[0], v[1][d] = s[1];
  }
}

}  // namespace
}  // namespace fp8q
