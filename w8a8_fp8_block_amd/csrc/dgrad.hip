// The gradient of the block-scaled projection's input on gfx950 (gemm_dgrad.h has the
// kernel's body):
//
//   dx[m,k] = sum_n dy[m,n] * w[n,k]
//
// The sum's index n runs along w's rows, in their forward layout: no transposed copy of
// the weights exists, their fragments come through the transposing LDS read.
#include "gemm_dgrad.h"
#include "launch.h"

namespace fp8q {
namespace {

template <int TM, bool SPLIT>
__global__ __launch_bounds__(256, 1) void dgrad_kernel(
    const uint8_t* __restrict__ dy, const float* __restrict__ dys, const uint8_t* __restrict__ w,
    const float* __restrict__ ws, uint16_t* __restrict__ dx, float* __restrict__ part, uint32_t M, uint32_t N,
    uint32_t K, uint32_t Mp, uint32_t tiles_m, uint32_t tiles_k, uint32_t splits) {
  using C = DgradCfg<TM>;
  uint32_t tmi, tki, split = 0;
  if constexpr (SPLIT)
    tile_split_coords(tiles_m, tiles_k, splits, tmi, tki, split);
  else
    tile_coords<C::GROUP>(tiles_m, tiles_k, tmi, tki);
  const uint32_t G = N / kGroup, b0 = SPLIT ? split * G / splits : 0;
  const uint32_t b1 = SPLIT ? (split + 1) * G / splits : G;
  gemm_dgrad_body<C, SPLIT>(dy, dys, w, ws, dx, part, tmi * C::BM, tki * C::BN, b0, b1 - b0, split, M, N, K, Mp);
}

template <int TM, bool SPLIT>
hipError_t launch(const uint8_t* dy, const float* dys, const uint8_t* w, const float* ws, uint16_t* dx, float* part,
                  uint32_t M, uint32_t N, uint32_t K, uint32_t splits, hipStream_t s) {
  using C = DgradCfg<TM>;
  const hipError_t e = allow_lds<&dgrad_kernel<TM, SPLIT>, C::LDS_BYTES>();
  if (e != hipSuccess) return e;
  const uint32_t tiles_m = (M + C::BM - 1) / C::BM, tiles_k = K / C::BN;
  dgrad_kernel<TM, SPLIT><<<dim3(tiles_m * tiles_k * splits), dim3(256), C::LDS_BYTES, s>>>(
      dy, dys, w, ws, dx, part, M, N, K, m_pad16(M), tiles_m, tiles_k, splits);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_dgrad(const uint8_t* dy, const float* dy_s_km, const uint8_t* w, const float* w_s, uint16_t* dx,
                             float* part, uint32_t M, uint32_t N, uint32_t K, bool wide, uint32_t splits,
                             hipStream_t s) {
  if (splits < 2)
    return wide ? launch<4, false>(dy, dy_s_km, w, w_s, dx, nullptr, M, N, K, 1, s)
                : launch<2, false>(dy, dy_s_km, w, w_s, dx, nullptr, M, N, K, 1, s);
  const hipError_t e = wide ? launch<4, true>(dy, dy_s_km, w, w_s, dx, part, M, N, K, splits, s)
                            : launch<2, true>(dy, dy_s_km, w, w_s, dx, part, M, N, K, splits, s);
  return e != hipSuccess ? e : launch_splitk_reduce(part, dx, M, K, splits, s);
}

}  // namespace fp8q
