// The gradient of the block-scaled projection's input on gfx950:
//
//   dx[m,k] = sum_n dy[m,n] * w[n,k]
//
// It is the forward GEMM's main loop (gemm_tile.h,
// gemm_pp.h) over the weights in their forward layout: the sum's index n runs
// along w's rows, and the weight fragments come through the transposing LDS read.
#include "gemm_pp.h"
#include "launch.h"

namespace fp8q {
namespace {

// In the bodies' terms the sum's length is N and the output's columns are K.
template <int STAGES, bool SPLIT>
__global__ __launch_bounds__(256, 2) void dgrad_tiled_kernel(
    const uint8_t* __restrict__ dy, const float* __restrict__ dys, const uint8_t* __restrict__ w,
    const float* __restrict__ ws, uint16_t* __restrict__ dx, uint32_t M, uint32_t N, uint32_t K, uint32_t Mp,
    uint32_t tiles_m, uint32_t tiles_n, uint32_t splits, float* __restrict__ part) {
  uint32_t tmi, tni, split = 0;
  if constexpr (SPLIT)
    tile_split_coords(tiles_m, tiles_n, splits, tmi, tni, split);
  else
    tile_coords(tiles_m, tiles_n, tmi, tni);
  gemm_tiled_body<128, 128, 2, 2, STAGES, false, SPLIT, DenseRows, NoEpilogue, 0, true>(
      dy, dys, w, ws, dx, tmi * 128, tni * 128, K, N, Mp, split, splits, part, DenseRows{M, M}, NoEpilogue{});
}

template <int STAGES, bool SPLIT>
hipError_t launch_dgrad_tiled(const uint8_t* dy, const float* dys, const uint8_t* w, const float* ws, uint16_t* dx,
                              float* part, uint32_t M, uint32_t N, uint32_t K, uint32_t splits, hipStream_t s) {
  using C = TileCfg<128, 128, 2, 2, STAGES>;
  const hipError_t e = allow_lds<&dgrad_tiled_kernel<STAGES, SPLIT>, C::LDS_BYTES>();
  if (e != hipSuccess) return e;
  const uint32_t tiles_m = (M + 127) / 128, tiles_n = K / 128;
  dgrad_tiled_kernel<STAGES, SPLIT><<<dim3(tiles_m * tiles_n * splits), dim3(C::NT), C::LDS_BYTES, s>>>(
      dy, dys, w, ws, dx, M, N, K, m_pad16(M), tiles_m, tiles_n, splits, part);
  return hipGetLastError();
}

__global__ __launch_bounds__(512) void dgrad_pp_kernel(
    const uint8_t* __restrict__ dy, const float* __restrict__ dys, const uint8_t* __restrict__ w,
    const float* __restrict__ ws, uint16_t* __restrict__ dx, uint32_t M, uint32_t N, uint32_t K, uint32_t Mp,
    uint32_t tiles_m, uint32_t tiles_n) {
  using C = PpCfg<3>;
  uint32_t tmi, tni;
  tile_coords(tiles_m, tiles_n, tmi, tni);
  gemm_pp_body<3, false, false, DenseRows, NoEpilogue, true>(dy, dys, w, ws, dx, tmi * C::BM, tni * C::BN, K, N, Mp,
                                                             FfnArgs{}, DenseRows{M, M}, NoEpilogue{});
}

hipError_t launch_dgrad_pp(const uint8_t* dy, const float* dys, const uint8_t* w, const float* ws, uint16_t* dx,
                           uint32_t M, uint32_t N, uint32_t K, hipStream_t s) {
  using C = PpCfg<3>;
  const hipError_t e = allow_lds<&dgrad_pp_kernel, C::LDS_BYTES>();
  if (e != hipSuccess) return e;
  const uint32_t tiles_m = (M + C::BM - 1) / C::BM, tiles_n = K / C::BN;
  dgrad_pp_kernel<<<dim3(tiles_m * tiles_n), dim3(C::NT), C::LDS_BYTES, s>>>(dy, dys, w, ws, dx, M, N, K, m_pad16(M),
                                                                             tiles_m, tiles_n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_dgrad(const uint8_t* dy, const float* dy_s_km, const uint8_t* w, const float* w_s, uint16_t* dx,
                             float* part, uint32_t M, uint32_t N, uint32_t K, uint32_t splits, int kernel,
                             uint32_t cus, hipStream_t s) {
  // three LDS stages where a grid leaves each workgroup its CU (as the forward's split form)
  const uint64_t wgs = (uint64_t)((M + 127) / 128) * (K / 128) * splits;
  if (splits >= 2) {
    const hipError_t e = wgs <= cus ? launch_dgrad_tiled<3, true>(dy, dy_s_km, w, w_s, dx, part, M, N, K, splits, s)
                                    : launch_dgrad_tiled<2, true>(dy, dy_s_km, w, w_s, dx, part, M, N, K, splits, s);
    return e != hipSuccess ? e : launch_splitk_reduce(part, dx, M, K, splits, s);
  }
  if (kernel == 5) return launch_dgrad_pp(dy, dy_s_km, w, w_s, dx, M, N, K, s);
  return wgs <= cus ? launch_dgrad_tiled<3, false>(dy, dy_s_km, w, w_s, dx, nullptr, M, N, K, 1, s)
                    : launch_dgrad_tiled<2, false>(dy, dy_s_km, w, w_s, dx, nullptr, M, N, K, 1, s);
}

}  // namespace fp8q
