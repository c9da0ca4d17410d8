// The weights' gradient dw[n,k] = sum over tokens m of dy[m,n] * x[m,k], both
// operands FP8 with one power of two per column and 128 tokens, both in their own
// row-major layout.
//
//   dw[n,k] = sum_b 2^(ey[b,n] + ex[b,k]) * sum_{m in block b} dec(dy[m,n]) * dec(x[m,k])
//
// The sum runs along the rows of both matrices, so their fragments come through
// the transposing LDS read (mfma_common.h) and no transposed copy exists.  The
// scales are the matrix instruction's own operands, a byte a lane: the partial
// products need no fp32 multiply of their own and accumulate in the instruction's
// accumulators (measured as exact as scaled fp32 additions: 1.5e-5 of the
// result's norm over 4608 tokens either way, the instruction's own rounding of a
// 128-deep sum).
//
// Workgroup tile BM (columns n of dy) x BN (columns k of x), panels of 128 columns
// x 128 tokens in LDS, a ring of STAGES.  Tokens past M lie past the buffer
// resources' ends and load as zeros.
#pragma once

#include "mfma_common.h"

namespace fp8q {
namespace {

struct WgradArgs {
  const uint8_t *dy, *x;     // codes [M,N], [M,K]
  const uint32_t *ey, *ex;   // [ceil(M/512)][N], [K]: four token blocks' bytes a dword
  uint16_t* out;             // [N,K] bf16
  float* part;               // SPLIT: [splits][N][K]
  uint32_t M, N, K, tiles_n, tiles_k, splits;
};

template <int BM, int BN, int WGM, int WGN, int STAGES_>
struct WgradCfg {
  static constexpr int STAGES = STAGES_;
  static constexpr int NW = WGM * WGN, NT = 64 * NW;
  static constexpr int WM = BM / WGM, WN = BN / WGN, TM = WM / 16, TN = WN / 16;
  static constexpr int PANEL = 128 * 128;
  static constexpr int DY_BYTES = BM / 128 * PANEL, X_BYTES = BN / 128 * PANEL;
  static constexpr int SC_M = (WM + 63) / 64, SC_N = (WN + 63) / 64;  // scale loads a wave
  static constexpr int SCW_BYTES = (SC_M + SC_N) * 256;
  static constexpr int STAGE_BYTES = DY_BYTES + X_BYTES + NW * SCW_BYTES;
  static constexpr int LDS_BYTES = STAGES * STAGE_BYTES;
  static constexpr int CH = (DY_BYTES + X_BYTES) / 1024 / NW;  // 1 KB loads a wave
  static constexpr int LOADS = CH + SC_M + SC_N;
  static_assert(WM % 64 == 0 && WN % 64 == 0 && BM % 128 == 0 && BN % 128 == 0, "tile");
  static_assert((DY_BYTES + X_BYTES) / 1024 % NW == 0 && LDS_BYTES <= 160 * 1024, "loads, LDS");
  static_assert((STAGES - 1) * LOADS < 64, "vmcnt range");
};

__device__ __forceinline__ v4f mfma_e4m3_128_scaled(const v8i& a, const v8i& b, const v4f& c, uint32_t ea, uint32_t eb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, (int)ea, 0, (int)eb);
}

// The tile n0.., k0.. over the token blocks b0 .. b0 + G - 1.
template <class C, bool SPLIT>
__device__ __forceinline__ void gemm_wgrad_body(const WgradArgs& a, uint32_t n0, uint32_t k0, uint32_t b0, uint32_t G,
                                                uint32_t wm, uint32_t wn, uint32_t split) {
  constexpr int TM = C::TM, TN = C::TN, STAGES = C::STAGES;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const uint32_t tid = threadIdx.x, lane = tid & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t M = a.M, N = a.N, K = a.K, packs = (M + 511) / 512;
  const __amdgpu_buffer_rsrc_t rY = make_rsrc(a.dy, M * N), rX = make_rsrc(a.x, M * K);
  const __amdgpu_buffer_rsrc_t rEy = make_rsrc(a.ey, packs * N * 4), rEx = make_rsrc(a.ex, packs * K * 4);

  // 1 KB chunk ch of a stage: 8 token rows of panel ch / 16 (dy's panels first)
  uint32_t off[C::CH], step[C::CH];
  bool is_y[C::CH];
#pragma unroll
  for (int j = 0; j < C::CH; ++j) {
    const uint32_t ch = wave * C::CH + j, panel = ch / 16, row = (ch % 16) * 8 + (lane >> 3);
    is_y[j] = panel < (uint32_t)(C::DY_BYTES / C::PANEL);
    const uint32_t ld = is_y[j] ? N : K;
    const uint32_t col = is_y[j] ? n0 + panel * 128 : k0 + (panel - C::DY_BYTES / C::PANEL) * 128;
    off[j] = row * ld + col + ((lane & 7) ^ swz_t(row)) * 16;
    step[j] = 128 * ld;
  }
  const uint32_t sc = C::DY_BYTES + C::X_BYTES + wave * C::SCW_BYTES;
  const uint32_t band_n = n0 + wm * C::WM, band_k = k0 + wn * C::WN;
  auto issue = [&](uint32_t b, uint32_t slot) {
    uint8_t* base = smem + slot * C::STAGE_BYTES;
#pragma unroll
    for (int j = 0; j < C::CH; ++j) dma16(is_y[j] ? rY : rX, off[j], b * step[j], base + (wave * C::CH + j) * 1024);
#pragma unroll
    for (int j = 0; j < C::SC_M; ++j) dma4(rEy, (band_n + j * 64 + lane) * 4, (b >> 2) * N * 4, base + sc + j * 256);
#pragma unroll
    for (int j = 0; j < C::SC_N; ++j)
      dma4(rEx, (band_k + j * 64 + lane) * 4, (b >> 2) * K * 4, base + sc + (C::SC_M + j) * 256);
  };

  const uint32_t l16 = lane & 15, lt = transposed_lane(lane);
  // fragment of the 16 columns col.. (of the operand's panels at `panels`)
  auto frag = [&](const uint8_t* panels, uint32_t col) -> v8i {
    const uint8_t* p = panels + col / 128 * C::PANEL + (lt ^ (col % 128));
    v8i f;
    f.lo = ld_transposed(p, 0);
    f.hi = ld_transposed(p, 1);
    return f;
  };

  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  if (G > 0) {
    const uint32_t last = b0 + G - 1;
#pragma unroll
    for (int s = 0; s < STAGES; ++s) issue(min(b0 + s, last), s);
    for (uint32_t i = 0; i < G; ++i) {
      const uint32_t slot = i % STAGES;
      const uint8_t* base = smem + slot * C::STAGE_BYTES;
      wait_vmcnt<(STAGES - 1) * C::LOADS>();
      wg_barrier();
      v8i fy[TM], fx[TN];
      uint32_t ey[TM], ex[TN];
      const uint32_t sh = 8 * ((b0 + i) & 3);
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        fy[t] = frag(base, wm * C::WM + t * 16);
        ey[t] = *reinterpret_cast<const uint32_t*>(base + sc + (t * 16 + l16) * 4) >> sh;
      }
#pragma unroll
      for (int t = 0; t < TN; ++t) {
        fx[t] = frag(base + C::DY_BYTES, wn * C::WN + t * 16);
        ex[t] = *reinterpret_cast<const uint32_t*>(base + sc + C::SC_M * 256 + (t * 16 + l16) * 4) >> sh;
      }
      wait_lgkm0();
      wg_barrier();  // every wave has read the slot
      issue(min(b0 + i + STAGES, last), slot);
#pragma unroll
      for (int i2 = 0; i2 < TM; ++i2)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i2][j] = mfma_e4m3_128_scaled(fx[j], fy[i2], acc[i2][j], ex[j], ey[i2]);
    }
    wait_vmcnt<0>();  // no direct load may still be writing LDS when the workgroup ends
  }
  // lane: row n = band + 16 i + l16, columns k = band + 16 j + 4 (lane / 16) ..
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const uint32_t n = band_n + i * 16 + l16;
    if (n < N) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const uint32_t k = band_k + j * 16 + 4 * (lane >> 4);
        if (k < K) {
          if constexpr (SPLIT)
            *reinterpret_cast<v4f*>(a.part + ((uint64_t)split * N + n) * K + k) = acc[i][j];
          else
            *reinterpret_cast<uint2*>(a.out + (uint64_t)n * K + k) = pack_bf16x4(acc[i][j]);
        }
      }
    }
  }
}

}  // namespace
}  // namespace fp8q
