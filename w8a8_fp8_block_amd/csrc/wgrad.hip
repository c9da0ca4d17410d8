// Launches of the weights' gradient (gemm_wgrad.h) on gfx950.
#include <algorithm>

#include "gemm_wgrad.h"
#include "launch.h"

namespace fp8q {
namespace {

using Wgrad256 = WgradCfg<4, 4>;
using Wgrad256x128 = WgradCfg<4, 2>;
using Wgrad128 = WgradCfg<2, 2>;

// Persistent workgroups, one a CU.  Each XCD has a contiguous run of the 256 x 256
// tiles (grouped order, so that its workgroups share operand panels in its L2) and
// deals them to its workgroups in turn.  Tiles left over for fewer than half or a
// quarter of the workgroups are cut in two or four, so that the last round costs its
// share.
__global__ __launch_bounds__(256, 1) void wgrad_kernel(WgradArgs a) {
  const uint32_t tiles = a.tiles_n * a.tiles_k;
  const uint32_t xcd = blockIdx.x & 7, worker = blockIdx.x >> 3, per = gridDim.x >> 3;
  const uint32_t q = tiles >> 3, r8 = tiles & 7;
  const uint32_t first = xcd * q + min(xcd, r8), count = q + (xcd < r8 ? 1 : 0);
  const uint32_t rounds = count / per, rest = count % per;
  const uint32_t pieces = rest * 4 <= per ? 4 : rest * 2 <= per ? 2 : 1;
  const uint32_t units = rounds + (pieces == 1 && worker < rest ? 1 : 0);
  auto tile = [&](uint32_t t, uint32_t& n0, uint32_t& k0) {
    grouped_tile(t, a.tiles_n, a.tiles_k, n0, k0);
    n0 *= 256;
    k0 *= 256;
  };
  if (units)
    gemm_wgrad_body<Wgrad256, false>(a, units, 0, a.M, 0, [&](uint32_t u, uint32_t& n0, uint32_t& k0) {
      tile(first + u * per + worker, n0, k0);
    });
  if (pieces > 1 && worker < rest * pieces) {
    uint32_t tn, tk;
    tile(first + rounds * per + worker / pieces, tn, tk);
    const uint32_t piece = worker % pieces;
    if (pieces == 2) {
      tk += piece * 128;
      if (tk < a.K)
        gemm_wgrad_body<Wgrad256x128, false>(a, 1, 0, a.M, 0, [&](uint32_t, uint32_t& n0, uint32_t& k0) {
          n0 = tn;
          k0 = tk;
        });
    } else {
      tn += piece / 2 * 128;
      tk += piece % 2 * 128;
      if (tn < a.N && tk < a.K)
        gemm_wgrad_body<Wgrad128, false>(a, 1, 0, a.M, 0, [&](uint32_t, uint32_t& n0, uint32_t& k0) {
          n0 = tn;
          k0 = tk;
        });
    }
  }
}

// Split form for few tiles: each 128 x 128 tile's token blocks cut into `splits`
// ranges, their fp32 sums to part; two workgroups share a CU.
__global__ __launch_bounds__(256, 2) void wgrad_split_kernel(WgradArgs a) {
  uint32_t tn, tk, split;
  tile_split_coords(a.tiles_n, a.tiles_k, a.splits, tn, tk, split);
  const uint32_t blocks = (a.M + 127) / 128;
  const uint32_t b0 = split * blocks / a.splits, b1 = (split + 1) * blocks / a.splits;
  gemm_wgrad_body<Wgrad128, true>(a, 1, 128 * b0, min(128 * b1, a.M), split, [&](uint32_t, uint32_t& n0, uint32_t& k0) {
    n0 = tn * 128;
    k0 = tk * 128;
  });
}

// dw of no tokens
__global__ __launch_bounds__(256) void wgrad_zero_kernel(uint4* out, uint64_t n) {
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (uint64_t)gridDim.x * 256)
    out[i] = make_uint4(0, 0, 0, 0);
}

}  // namespace

hipError_t launch_gemm_wgrad(const uint8_t* dy, const uint8_t* ey, const uint8_t* x, const uint8_t* ex, uint16_t* dw,
                             float* part, uint32_t M, uint32_t N, uint32_t K, uint32_t splits, uint32_t cus,
                             hipStream_t s) {
  if (M == 0) {
    const uint64_t n = (uint64_t)N * K / 8;
    wgrad_zero_kernel<<<dim3((uint32_t)std::min<uint64_t>((n + 255) / 256, 2048)), dim3(256), 0, s>>>(
        reinterpret_cast<uint4*>(dw), n);
    return hipGetLastError();
  }
  WgradArgs a{dy, x, reinterpret_cast<const uint32_t*>(ey), reinterpret_cast<const uint32_t*>(ex), dw, part,
              M,  N, K, 0, 0, splits};
  if (splits >= 2) {
    const hipError_t e = allow_lds<&wgrad_split_kernel, Wgrad128::LDS_BYTES>();
    if (e != hipSuccess) return e;
    a.tiles_n = N / 128;
    a.tiles_k = K / 128;
    wgrad_split_kernel<<<dim3(a.tiles_n * a.tiles_k * splits), dim3(256), Wgrad128::LDS_BYTES, s>>>(a);
    const hipError_t l = hipGetLastError();
    return l != hipSuccess ? l : launch_splitk_reduce(part, dw, N, K, splits, s);
  }
  const hipError_t e = allow_lds<&wgrad_kernel, Wgrad256::LDS_BYTES>();
  if (e != hipSuccess) return e;
  a.tiles_n = (N + 255) / 256;
  a.tiles_k = (K + 255) / 256;
  wgrad_kernel<<<dim3(std::max(cus / 8, 1u) * 8), dim3(256), Wgrad256::LDS_BYTES, s>>>(a);
  return hipGetLastError();
}

}  // namespace fp8q
