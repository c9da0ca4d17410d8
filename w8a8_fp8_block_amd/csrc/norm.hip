// RMS norm with the residual's addition and FP8 output, and its gradient, for
// gfx950.
//
//   h    = bf16(x + r)                     (h = x where there is no residual)
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y    = h * rstd * w                    (fp32)
//   per (token, 128 columns): scale = amax|y| / 448, q = e4m3(y / scale)
//
// h is rounded to bf16 before it is normalised: it is the residual stream that
// the next layer and the gradient read, so all of them see one value.  y is
// quantized from fp32 (one rounding, to 8 bits); the bf16 copy of y, for
// consumers that take bf16, is rounded by itself.  Sums and statistics are fp32.
//
// The gradient, with g = w * dy and xhat = h * rstd:
//   dx = dh + rstd * (g - xhat * mean(g * xhat)),   dw = sum over rows of dy * xhat
//
// Both are bound by memory: each element is loaded once into registers, reduced
// over the row and finished from there.  A row belongs to W waves, lane t
// holding the 8-value chunks t, t + 64 W, ...: 16 consecutive lanes hold a scale
// group, whose maximum is one DPP reduction.  4576 x 5120, inputs from HBM: 39 us with
// residual and bf16 copy (211 MB, 5.4 TB/s; a copy of 1 GiB moves 5.1), the gradient 42 us
// (187 MB), 39 of them in its first kernel; one token of 5120: 2.7 us, an empty launch's 2.3.
#include <algorithm>

#include "wave_common.h"

namespace fp8q {
namespace {

// Scale and quotients of N of a group's fp32 values, from its maximum's bits:
//   s = fl(amax / 448),  q = fl(y / s), at most 448 in magnitude (e4m3's saturation).
// fl(a / 448) by a corrected product and the quotients by reciprocal are the correctly
// rounded ones where s is normal.  (Of all finite a, those up to 2^-120 alone give another
// scale.  Of all mantissas of s, with y on both sides of every border between two codes, the
// last one alone gives a quotient that rounds to another code, at y / s = 2^-10 and only if
// the hardware reciprocal is off by an ulp there; it is divided out too.  From s = 2^-80 the
// residuals of quotients down to 2^-11, the least that matter, are exact.)  Other
// scales - zero, tiny, infinite, NaN - are divided out.  The choice is uniform over the
// wave and both ways give the same codes, so a group's do not depend on its neighbours.
// Only a subnormal scale, a few units of 2^-149, rounds so far that y / s passes 448: by up
// to 224 / 448, beyond what the conversion saturates by itself (it would give NaN).
template <int N>
__device__ __forceinline__ float scale_and_quotients(const float* y, uint32_t amax_bits, float* q) {
  const float a = __uint_as_float(amax_bits);
  constexpr float k = 1.0f / 448.0f;
  const float s0 = a * k;
  float s = __builtin_fmaf(-__builtin_fmaf(s0, 448.0f, -a), k, s0);
  const bool slow = !(s >= 0x1p-80f && s < INFINITY) || (__float_as_uint(s) & 0x7FFFFFu) == 0x7FFFFFu;
  if (__builtin_amdgcn_ballot_w64(slow) == 0) {
    quotients_by_reciprocal<N>(y, s, q);
  } else {
    s = a / 448.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float v = s == 0.0f ? y[i] : y[i] / s;
      q[i] = v > 448.0f ? 448.0f : v < -448.0f ? -448.0f : v;  // a NaN stays one
    }
  }
  return s;
}

// 1 / sqrt(v), v normal: the hardware's (1 ulp) and one Newton step; NaN for v
// infinite (the square sum left fp32's range).
__device__ __forceinline__ float rsqrt_f32(float v) {
  const float r = __builtin_amdgcn_rsqf(v);
  return __builtin_fmaf(r * 0.5f, __builtin_fmaf(-v * r, r, 1.0f), r);
}

// Sum over the W waves of this wave's row; red: one float a wave.  Called by the
// whole workgroup; the next call must use the other half of a double buffer.
template <uint32_t W>
__device__ __forceinline__ float row_sum(float v, float* red, uint32_t wave) {
  v = wave_sum_f32(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    const uint32_t first = wave / W * W;
    v = red[first];
#pragma unroll
    for (uint32_t i = 1; i < W; ++i) v += red[first + i];
  }
  return v;
}

struct NormArgs {
  const u32x4 *x, *r, *w;  // r NULL: no residual
  u32x4 *h, *y;            // either may be NULL
  u32x2* q;
  float *srm, *skm, *rstd;  // any may be NULL
  float eps;
  uint32_t M, K, Mp;
};

constexpr uint32_t kNormMaxWaves = 16;

// W waves a row, C chunks a lane; blockDim.x / (64 W) rows a workgroup.
template <uint32_t W, uint32_t C>
__global__ __launch_bounds__(1024) void norm_quant_kernel(NormArgs a) {
  extern __shared__ float scales[];  // [rows][G]: the K-major scales' staging
  __shared__ float red[kNormMaxWaves];
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t rows = (blockDim.x >> 6) / W, row = wave / W;
  const uint32_t m0 = blockIdx.x * rows, m = m0 + row;
  const uint32_t t = (wave % W) * 64 + lane, chunks = a.K / 8, G = a.K / kGroup;
  const bool live = m < a.M;
  const uint64_t base = (uint64_t)m * chunks;

  // every load of the row before the first store (h may be x's or r's own array)
  u32x4 h[C];
#pragma unroll
  for (uint32_t i = 0; i < C; ++i) {
    const uint32_t c = t + 64 * W * i;
    h[i] = u32x4{0, 0, 0, 0};
    if (live && c < chunks) h[i] = __builtin_nontemporal_load(&a.x[base + c]);
  }
  if (a.r) {
    u32x4 r[C];
#pragma unroll
    for (uint32_t i = 0; i < C; ++i) {
      const uint32_t c = t + 64 * W * i;
      r[i] = u32x4{0, 0, 0, 0};
      if (live && c < chunks) r[i] = __builtin_nontemporal_load(&a.r[base + c]);
    }
#pragma unroll
    for (uint32_t i = 0; i < C; ++i) {
      const uint32_t c = t + 64 * W * i;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[i][j] = bf16x2_rne(bf_lo(h[i][j]) + bf_lo(r[i][j]), bf_hi(h[i][j]) + bf_hi(r[i][j]));
      if (live && c < chunks) __builtin_nontemporal_store(h[i], &a.h[base + c]);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (uint32_t i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ss = __builtin_fmaf(bf_lo(h[i][j]), bf_lo(h[i][j]), ss);
      ss = __builtin_fmaf(bf_hi(h[i][j]), bf_hi(h[i][j]), ss);
    }
  ss = row_sum<W>(ss, red, wave);
  const float rstd = rsqrt_f32(ss / (float)a.K + a.eps);
  if (live && t == 0 && a.rstd) a.rstd[m] = rstd;

#pragma unroll
  for (uint32_t i = 0; i < C; ++i) {
    const uint32_t c = t + 64 * W * i;
    if (live && c < chunks) {  // uniform over a group's 16 lanes
      const u32x4 w = a.w[c];
      float y[8], qv[8];
      uint32_t amax = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[2 * j] = bf_lo(h[i][j]) * rstd * bf_lo(w[j]);
        y[2 * j + 1] = bf_hi(h[i][j]) * rstd * bf_hi(w[j]);
        amax = max(amax, max(__float_as_uint(y[2 * j]) & 0x7FFFFFFFu, __float_as_uint(y[2 * j + 1]) & 0x7FFFFFFFu));
      }
      amax = dpp_row_max_u32(amax);
      const float s = scale_and_quotients<8>(y, amax, qv);
      a.q[base + c] = u32x2{encode4(qv), encode4(qv + 4)};
      if (a.y) {
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = bf16x2_rne(y[2 * j], y[2 * j + 1]);
        __builtin_nontemporal_store(o, &a.y[base + c]);
      }
      if ((lane & 15) == 0) {
        if (a.srm) a.srm[(uint64_t)m * G + c / 16] = s;
        scales[row * G + c / 16] = s;
      }
    }
  }
  if (a.skm) {
    // the K-major scales of the workgroup's rows, runs of `rows` along the
    // tokens; the last workgroup writes the pad slots too
    __syncthreads();
    const uint32_t end = m0 + rows >= a.M ? a.Mp - m0 : rows;
    for (uint32_t i = threadIdx.x; i < G * end; i += blockDim.x) {
      const uint32_t g = i / end, r = i % end;
      a.skm[(uint64_t)g * a.Mp + m0 + r] = m0 + r < a.M ? scales[r * G + g] : 0.0f;
    }
  }
}

struct NormGradArgs {
  const u32x4 *dy, *dh, *h, *w;  // dh may be NULL
  const float* rstd;
  u32x4* dx;
  float* part;  // [gridDim.x][K]
  uint32_t M, K;
};

// Row groups of W waves take the rows g, g + groups, ... and keep their share of dw in
// registers; the row groups of a workgroup (blockDim.x / (64 W)) meet in LDS at the end.
// T: the workgroup's threads at most.  (dh loaded behind the row's sum where a lane holds
// three chunks or four: 4576 x 17408 131 us, with the other loads 165.  128 registers a lane do
// not hold three or four chunks of it all: a few spill at three, 40 of them at four, where 2000
// x 32768 takes 209 us, 2.5 TB/s.)
template <uint32_t W, uint32_t C, uint32_t T>
__global__ __launch_bounds__(T) void norm_grad_kernel(NormGradArgs a) {
  extern __shared__ float dws[];  // [K], where a workgroup holds several row groups
  __shared__ float red[2][kNormMaxWaves];
  const uint32_t wave = threadIdx.x >> 6, rows = (blockDim.x >> 6) / W, row = wave / W;
  const uint32_t t = threadIdx.x % (64 * W), chunks = a.K / 8;
  const float inv_k = 1.0f / (float)a.K;

  float dw[C][8];
#pragma unroll
  for (uint32_t i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  uint32_t turn = 0;
  for (uint64_t m0 = blockIdx.x * rows; m0 < a.M; m0 += gridDim.x * rows, turn ^= 1) {  // uniform
    const uint32_t m = (uint32_t)m0 + row;
    const bool live = m < a.M;
    const uint64_t base = (uint64_t)m * chunks;
    const float rstd = live ? a.rstd[m] : 0.0f;
    u32x4 dy[C], h[C], d[C];
#pragma unroll
    for (uint32_t i = 0; i < C; ++i) {
      const uint32_t c = t + 64 * W * i;
      dy[i] = h[i] = d[i] = u32x4{0, 0, 0, 0};
      if (live && c < chunks) {
        dy[i] = __builtin_nontemporal_load(&a.dy[base + c]);
        h[i] = __builtin_nontemporal_load(&a.h[base + c]);
        if (C <= 2 && a.dh) d[i] = __builtin_nontemporal_load(&a.dh[base + c]);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < C; ++i) {
      const uint32_t c = t + 64 * W * i;
      const u32x4 w = c < chunks ? a.w[c] : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float l = bf_lo(dy[i][j]) * (bf_lo(h[i][j]) * rstd), u = bf_hi(dy[i][j]) * (bf_hi(h[i][j]) * rstd);
        dw[i][2 * j] += l;
        dw[i][2 * j + 1] += u;
        s = __builtin_fmaf(l, bf_lo(w[j]), s);
        s = __builtin_fmaf(u, bf_hi(w[j]), s);
      }
    }
    s = row_sum<W>(s, red[turn], wave) * inv_k;
#pragma unroll
    for (uint32_t i = 0; i < C; ++i) {
      const uint32_t c = t + 64 * W * i;
      if (live && c < chunks) {
        const u32x4 w = a.w[c];
        if (C > 2 && a.dh) d[i] = __builtin_nontemporal_load(&a.dh[base + c]);  // (sooner, more registers spill)
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float l = rstd * (bf_lo(dy[i][j]) * bf_lo(w[j]) - bf_lo(h[i][j]) * rstd * s);
          const float u = rstd * (bf_hi(dy[i][j]) * bf_hi(w[j]) - bf_hi(h[i][j]) * rstd * s);
          o[j] = bf16x2_rne(l + bf_lo(d[i][j]), u + bf_hi(d[i][j]));
        }
        __builtin_nontemporal_store(o, &a.dx[base + c]);
      }
    }
  }
  float* out = a.part + (uint64_t)blockIdx.x * a.K;
  for (uint32_t r = 0; r < rows; ++r) {  // the row groups in order; the last one writes
    if (r) __syncthreads();
    if (row == r) {
#pragma unroll
      for (uint32_t i = 0; i < C; ++i) {
        const uint32_t c = t + 64 * W * i;
        if (c < chunks) {
          float4* o = reinterpret_cast<float4*>((r + 1 == rows ? out : dws) + 8 * c);
          float4 lo = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
          float4 hi = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
          if (r) {
            const float4* b = reinterpret_cast<const float4*>(dws + 8 * c);
            lo.x += b[0].x, lo.y += b[0].y, lo.z += b[0].z, lo.w += b[0].w;
            hi.x += b[1].x, hi.y += b[1].y, hi.z += b[1].z, hi.w += b[1].w;
          }
          o[0] = lo;
          o[1] = hi;
        }
      }
    }
  }
}

// dw[k] = sum of the parts, 16 waves taking each 16th one, then in wave order.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                       uint32_t parts, uint32_t K) {
  __shared__ float sum[16][64];
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, k = blockIdx.x * 64 + lane;
  float s = 0.0f;
  for (uint32_t p0 = wave; p0 < parts; p0 += 128) {  // eight loads in flight
    float v[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) v[i] = p0 + 16 * i < parts ? part[(uint64_t)(p0 + 16 * i) * K + k] : 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) s += v[i];
  }
  sum[wave][lane] = s;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int w = 1; w < 16; ++w) s += sum[w][lane];
    dw[k] = s;
  }
}

// Waves that a row takes, of those below: the fewest whose lanes hold it in `most` chunks
// each, or 16.
constexpr uint32_t kRowWaves[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16};
uint32_t row_waves(uint32_t K, uint32_t most) {
  for (uint32_t w : kRowWaves)
    if (K / 8 <= 64 * w * most) return w;
  return 16;
}

// f(W, C) for a row's waves and chunks a lane
template <class F>
hipError_t for_row(uint32_t K, uint32_t most, F&& f) {
  using std::integral_constant;
  const uint32_t w = row_waves(K, most), c = (K / 8 + 64 * w - 1) / (64 * w);
  auto chunks = [&](auto W) -> hipError_t {
    if (c <= 1) return f(W, integral_constant<uint32_t, 1>{});
    if (c <= 2) return f(W, integral_constant<uint32_t, 2>{});
    if constexpr (decltype(W)::value == 16) {
      if (c <= 3) return f(W, integral_constant<uint32_t, 3>{});
      if (c <= 4) return f(W, integral_constant<uint32_t, 4>{});
    }
    return hipErrorInvalidValue;
  };
  switch (w) {
    case 1: return chunks(integral_constant<uint32_t, 1>{});
    case 2: return chunks(integral_constant<uint32_t, 2>{});
    case 3: return chunks(integral_constant<uint32_t, 3>{});
    case 4: return chunks(integral_constant<uint32_t, 4>{});
    case 5: return chunks(integral_constant<uint32_t, 5>{});
    case 6: return chunks(integral_constant<uint32_t, 6>{});
    case 8: return chunks(integral_constant<uint32_t, 8>{});
    case 10: return chunks(integral_constant<uint32_t, 10>{});
    case 12: return chunks(integral_constant<uint32_t, 12>{});
    default: return chunks(integral_constant<uint32_t, 16>{});
  }
}

// Row groups of a workgroup, about 12 waves
constexpr uint32_t group_rows(uint32_t W) { return W >= 8 ? 1 : 12 / W; }

// Up to this many rows each has a workgroup and twice the waves (5120 columns, us without ->
// with: 3.7 -> 3.3 at one row, 4.5 -> 3.6 at 25, 5.7 -> 4.8 at 256; equal from 409.  The
// gradient: 6.9 -> 6.2 at 64, 8.6 -> 8.1 at 200; 10.6 -> 11.0 at 409).
constexpr uint32_t kNormFewRows = 256;
// Workgroups of a gradient call: one a CU (256 CUs).  At most 128 / 256 / 512, us in a graph: 11.8
// / 11.5 / 11.5 at 512 x 6144 (256 workgroups' rows), 19.9 / 17.6 / 19.4 at 1168 x 6144, 13.0 /
// 11.7 / 14.5 at 4576 x 640, 47.9 / 35.0 / 38.0 at 4576 x 5120.
constexpr uint32_t kNormGradParts = 256;
// A gradient call that one workgroup does in two turns at most writes dw itself, one launch and
// not two.  In one turn that saves time on both sides; the second turn saves it on the host
// and costs some on the device.  us a call from the host / in a graph, two launches -> one:
// one turn: 8 x 384 8.5 -> 6.0 / 4.2 -> 3.6, 2 x 5120 8.5 -> 6.0 / 5.0 -> 3.8; two turns: 24 x 384 9.7
// -> 6.8 / 4.1 -> 4.5, 12 x 2048 9.5 -> 6.6 / 4.5 -> 5.7 (the worst), 4 x 5120 9.9 -> 6.8 / 4.9 -> 5.1,
// 2 x 17408 9.8 -> 7.1 / 7.5 -> 7.1.
bool norm_grad_lone(uint32_t M, uint32_t K) { return M > 0 && M <= 2 * group_rows(row_waves(K, 2)); }
uint32_t norm_grad_parts(uint32_t M, uint32_t K) {
  if (norm_grad_lone(M, K)) return 1;
  if (M <= kNormFewRows) return M;
  const uint32_t rows = group_rows(row_waves(K, 2));
  return std::min((M + rows - 1) / rows, kNormGradParts);
}

}  // namespace

hipError_t launch_norm_quant(const uint16_t* x, const uint16_t* r, const uint16_t* w, uint16_t* h, uint16_t* y,
                             uint8_t* q, float* scale_rm, float* scale_km, float* rstd, float eps, uint32_t M,
                             uint32_t K, hipStream_t s) {
  const NormArgs a{reinterpret_cast<const u32x4*>(x), reinterpret_cast<const u32x4*>(r),
                   reinterpret_cast<const u32x4*>(w), reinterpret_cast<u32x4*>(h), reinterpret_cast<u32x4*>(y),
                   reinterpret_cast<u32x2*>(q), scale_rm, scale_km, rstd, eps, M, K, m_pad16(M)};
  return for_row(K, M <= kNormFewRows ? 1 : 2, [&](auto W, auto C) {
    const uint32_t rows = M <= kNormFewRows ? 1 : group_rows(W);
    norm_quant_kernel<W, C><<<dim3((M + rows - 1) / rows), dim3(64 * W * rows), rows * (K / kGroup) * 4, s>>>(a);
    return hipGetLastError();
  });
}

uint64_t norm_grad_workspace_bytes(uint32_t M, uint32_t K) {
  return (uint64_t)norm_grad_parts(M, K) * K * 4;
}

hipError_t launch_norm_grad(const uint16_t* dy, const uint16_t* dh, const uint16_t* h, const uint16_t* w,
                            const float* rstd, uint16_t* dx, float* dw, void* workspace, uint32_t M, uint32_t K,
                            hipStream_t s) {
  const bool lone = norm_grad_lone(M, K), few = !lone && M <= kNormFewRows;
  const uint32_t parts = norm_grad_parts(M, K);
  const NormGradArgs a{reinterpret_cast<const u32x4*>(dy), reinterpret_cast<const u32x4*>(dh),
                       reinterpret_cast<const u32x4*>(h), reinterpret_cast<const u32x4*>(w), rstd,
                       reinterpret_cast<u32x4*>(dx), lone ? dw : static_cast<float*>(workspace), M, K};
  if (M > 0) {
    const hipError_t e = for_row(K, few ? 1 : 2, [&](auto W, auto C) {
      if (few) {
        norm_grad_kernel<W, C, 64 * W><<<dim3(parts), dim3(64 * W), 0, s>>>(a);
      } else {
        constexpr uint32_t rows = group_rows(W);
        norm_grad_kernel<W, C, 64 * W * rows><<<dim3(parts), dim3(64 * W * rows), rows > 1 ? K * 4 : 0, s>>>(a);
      }
      return hipGetLastError();
    });
    if (e != hipSuccess || lone) return e;
  }
  norm_dw_kernel<<<dim3(K / 64), dim3(1024), 0, s>>>(a.part, dw, parts, K);
  return hipGetLastError();
}

}  // namespace fp8q
