// Two-way FP8 quantizer for gfx950: one pass over a bf16 matrix x [M,K] gives the
// codes that a product over its columns reads and those that a product over its
// rows (the tokens) reads.
//
//   rows:    per (row, 128 columns)  scale = amax/448 (fp32),  q = e4m3(x / scale),
//            the activation quantizer's own steps (quant_common.h)
//   tokens:  per (128 rows, column)  2^e, the least e with amax <= 448 * 2^e
//            (e >= -127),  q_tok = e4m3(x / 2^e), kept as the byte e + 127
//
// The token scales are powers of two because the matrix instruction then applies
// them itself (gemm_wgrad.h); x / 2^e is exact, so q_tok rounds once.  Its codes
// stay in x's own layout: the product's transposing LDS reads take them as they
// are, and no transposed copy is written.
//
// Bound by memory.  A workgroup holds a 128 x 128 tile in registers, 16 lanes a
// row, 8 columns and 8 rows a thread; a row's maximum is one DPP reduction, a
// column's goes through a shuffle and LDS.  Five waves a SIMD, so that other tiles' loads
// lie over a tile's two reductions.  4576 x 17408 with both codes, from HBM: 59.5 us (319 MB,
// 5.4 TB/s; a copy of 1 GiB moves 5.1); 409 x 1408, tokens alone: 3.8 us, a launch's 2.3 and
// one chain of load, reduction and store.
#include "quant_common.h"

namespace fp8q {
namespace {

constexpr uint32_t kDualThreads = 256, kDualRows = 8;  // rows a thread: r0 + 16 i

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(as_u16x2(a), as_u16x2(b)));
}

// Byte e + 127 of a column's bf16 magnitude maximum: 448 = 1.75 * 2^8, so the
// exponent less 8, and one more where the mantissa is above 1.75.  NaN and
// infinity give 255, the scale that stands for NaN.
__device__ __forceinline__ uint32_t token_byte(uint32_t amax) {
  const int e = (int)(amax >> 7) - 8 + ((amax & 127u) > 96u ? 1 : 0);
  return amax >= 0x7F80u ? 255u : (uint32_t)max(e, 0);
}

template <bool ROWS>
__global__ __launch_bounds__(kDualThreads, 5) void quant_dual_kernel(
    const u32x4* __restrict__ x, u32x2* __restrict__ q, float* __restrict__ skm, u32x2* __restrict__ qt,
    uint8_t* __restrict__ et, uint32_t M, uint32_t K, uint32_t Mp, uint32_t gtiles) {
  __shared__ uint32_t cmax[4][16][4];
  __shared__ float rscale[128];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t mb = blockIdx.x / gtiles, g = blockIdx.x % gtiles, m0 = mb * 128;
  const uint32_t c = tid & 15, r0 = tid >> 4, chunks = K / 8;

  u32x4 v[kDualRows];
#pragma unroll
  for (uint32_t i = 0; i < kDualRows; ++i) {
    const uint32_t m = m0 + r0 + 16 * i;
    v[i] = u32x4{0, 0, 0, 0};
    if (m < M) v[i] = __builtin_nontemporal_load(&x[(uint64_t)m * chunks + g * 16 + c]);
  }
  // column maxima: this thread's rows, the wave's, the workgroup's
  const uint32_t mag = 0x7FFF7FFFu;
  uint32_t cm[4] = {0, 0, 0, 0};
#pragma unroll
  for (uint32_t i = 0; i < kDualRows; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) cm[j] = max_u16x2(cm[j], v[i][j] & mag);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    cm[j] = max_u16x2(cm[j], (uint32_t)__shfl_xor((int)cm[j], 16));
    cm[j] = max_u16x2(cm[j], (uint32_t)__shfl_xor((int)cm[j], 32));
  }
  if (lane < 16) *reinterpret_cast<uint4*>(cmax[wave][c]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);

  if constexpr (ROWS) {
#pragma unroll
    for (uint32_t i = 0; i < kDualRows; ++i) {
      const uint32_t m = m0 + r0 + 16 * i;
      float s;
      const u32x2 codes = quant_group(v[i], s);
      if (m < M) __builtin_nontemporal_store(codes, &q[(uint64_t)m * chunks + g * 16 + c]);
      if (c == 0) rscale[r0 + 16 * i] = s;  // rows past M: zero, the pad slots' value
    }
  }
  __syncthreads();
#pragma unroll
  for (uint32_t w = 0; w < 4; ++w) {
    const uint4 o = *reinterpret_cast<const uint4*>(cmax[w][c]);
    cm[0] = max_u16x2(cm[0], o.x);
    cm[1] = max_u16x2(cm[1], o.y);
    cm[2] = max_u16x2(cm[2], o.z);
    cm[3] = max_u16x2(cm[3], o.w);
  }
  uint32_t b[8];
  float f[8];  // 2^-e
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    b[j] = token_byte((cm[j / 2] >> (16 * (j & 1))) & 0xFFFFu);
    f[j] = __uint_as_float((254u - min(b[j], 254u)) << 23);
  }
#pragma unroll
  for (uint32_t i = 0; i < kDualRows; ++i) {
    const uint32_t m = m0 + r0 + 16 * i;
    if (m < M) {
      float p[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[2 * j] = bf_lo(v[i][j]) * f[2 * j];
        p[2 * j + 1] = bf_hi(v[i][j]) * f[2 * j + 1];
      }
      __builtin_nontemporal_store(u32x2{encode4(p), encode4(p + 4)}, &qt[(uint64_t)m * chunks + g * 16 + c]);
    }
  }
  if (r0 == 0) {
    // this block's byte of each column's dword; the last block writes the bytes
    // past it as well
    const uint32_t last = m0 + 128 >= M ? 4 : (mb & 3) + 1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint8_t* o = et + ((uint64_t)(mb >> 2) * K + g * 128 + 8 * c + j) * 4;
      o[mb & 3] = (uint8_t)b[j];
      for (uint32_t p = (mb & 3) + 1; p < last; ++p) o[p] = 0;
    }
  }
  if constexpr (ROWS) {
    if (tid < 128 && m0 + tid < Mp) skm[(uint64_t)g * Mp + m0 + tid] = rscale[tid];
  }
}

}  // namespace

hipError_t launch_quant_dual(const uint16_t* x, uint8_t* q, float* scale_km, uint8_t* q_tok, uint8_t* exp_tok,
                             uint32_t M, uint32_t K, hipStream_t s) {
  const uint32_t gtiles = K / kGroup;
  const dim3 grid((M + 127) / 128 * gtiles), block(kDualThreads);
  const auto* xv = reinterpret_cast<const u32x4*>(x);
  if (q)
    quant_dual_kernel<true><<<grid, block, 0, s>>>(xv, reinterpret_cast<u32x2*>(q), scale_km,
                                                   reinterpret_cast<u32x2*>(q_tok), exp_tok, M, K, m_pad16(M), gtiles);
  else
    quant_dual_kernel<false><<<grid, block, 0, s>>>(xv, nullptr, nullptr, reinterpret_cast<u32x2*>(q_tok), exp_tok, M,
                                                    K, m_pad16(M), gtiles);
  return hipGetLastError();
}

}  // namespace fp8q
