// Statements of the skinny kernel (described in gemm_skinny.h), included in the body of
// gemm_skinny_kernel and of gemm_skinny_body.  As an inlined call the compiler
// waits for weight loads between the others of a K block where the columns' tail
// is loaded: 27.4 us instead of 26.5 at M = 96, N = 6144, K = 5120.  Uses the
// function's parameters and `epi`; no include guard.
  static_assert(!(SPLIT && ROW), "split form for block-scaled weights only");
  // partial sums of the waves (dynamic LDS: NWV*TN*TM KB)
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  v4f(*red)[TN][TM][64] = reinterpret_cast<v4f(*)[TN][TM][64]>(smem);
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w = blockIdx.x;
  // this workgroup's columns, in units of 4
  const uint32_t c0 = 4 * (w * units_base + min(w, units_rem));
  const uint32_t c1 = c0 + 4 * (units_base + (w < units_rem ? 1u : 0u));
  const uint32_t nt = (c1 - c0 + 15) / 16;
  const uint32_t G = K / kGroup;
  const uint32_t l16 = lane & 15, kq = 32 * (lane >> 4);  // this lane's byte offset in a K block
  // operand rows: weight row c0 + 16t + l16 (zero beyond c1), activation row 16tm + l16
  const uint8_t* wrow[TN];
  bool wok[TN];
  uint32_t wsi[TN];  // weight-scale row of this lane's four output columns
#pragma unroll
  for (int t = 0; t < TN; ++t) {
    const uint32_t r = c0 + 16 * t + l16;
    wok[t] = r < c1;
    wrow[t] = W + (uint64_t)min(r, N - 1) * K + kq;
    wsi[t] = min(c0 + 16 * t + 4 * (lane >> 4), N - 1) / kGroup * G;
  }
  const uint32_t m0 = blockIdx.y * (16 * TM);  // this workgroup's rows
  const uint8_t* arow[TM];
  uint32_t srow[TM];
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const uint32_t m = m0 + tm * 16 + l16;
    arow[tm] = A + (uint64_t)min(m, M - 1) * K + kq;
    srow[tm] = min(m, Mp - 1);
  }

  v4f acc[TN][TM];
#pragma unroll
  for (int t = 0; t < TN; ++t)
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) acc[t][tm] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // this workgroup's K blocks [kbeg, kend): all of them, or split z's range
  const uint32_t kbeg = SPLIT ? blockIdx.z * G / gridDim.z : 0;
  const uint32_t kend = SPLIT ? (blockIdx.z + 1) * G / gridDim.z : G;
  for (uint32_t kb0 = kbeg + wave; kb0 < kend; kb0 += NWV * U) {
    v8i wf[U][TN], af[U][TM];
    float as[U][TM], ws[U][TN];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t k = kb0 + u * NWV;
      if (k < kend) {
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          if ((uint32_t)t < nt) {
            if (wok[t]) {
              const u32x4* wp = reinterpret_cast<const u32x4*>(wrow[t] + (uint64_t)k * kGroup);
              wf[u][t] = join(__builtin_nontemporal_load(wp), __builtin_nontemporal_load(wp + 1));
            } else {
              wf[u][t] = v8i{0, 0, 0, 0, 0, 0, 0, 0};
            }
            ws[u][t] = ROW ? 1.0f : Ws[wsi[t] + k];
          }
        }
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
          const u32x4* ap = reinterpret_cast<const u32x4*>(arow[tm] + (uint64_t)k * kGroup);
          af[u][tm] = join(ap[0], ap[1]);
          as[u][tm] = As[(uint64_t)k * Mp + srow[tm]];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb0 + u * NWV < kend) {
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          if ((uint32_t)t < nt) {
#pragma unroll
            for (int tm = 0; tm < TM; ++tm) {
              const v4f p = mfma_e4m3_128(wf[u][t], af[u][tm]);
              acc[t][tm] += p * (as[u][tm] * ws[u][t]);
            }
          }
        }
      }
    }
  }

  epi.template add_shared<TM, TN, 64 * NWV>([&](int tm, int t) -> v4f& { return acc[t][tm]; }, smem, m0, c0, M,
                                            lane, SPLIT ? blockIdx.z * NWV + wave : wave,
                                            SPLIT ? NWV * gridDim.z : NWV);
#pragma unroll
  for (int t = 0; t < TN; ++t)
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) red[wave][t][tm][lane] = acc[t][tm];
  __syncthreads();
  // waves share the final sums: wave v sums and stores tiles (t, tm) with
  // t*TM + tm = v (mod NWV)
#pragma unroll
  for (int j = 0; j < TN * TM; ++j) {
    const int t = j / TM, tm = j % TM;
    if ((uint32_t)(j % NWV) == wave && (uint32_t)t < nt) {
      v4f s = red[0][t][tm][lane];
#pragma unroll
      for (int v = 1; v < NWV; ++v) s += red[v][t][tm][lane];
      const uint32_t m = m0 + tm * 16 + l16;
      const uint32_t n = c0 + 16 * t + 4 * (lane >> 4);
      if constexpr (ROW) {
        if (n < c1) {
          const float4 r = *reinterpret_cast<const float4*>(Ws + n);
          s *= v4f{r.x, r.y, r.z, r.w};
        }
      }
      if (m < M && n < c1) {
        if constexpr (SPLIT)
          *reinterpret_cast<v4f*>(part + ((uint64_t)blockIdx.z * M + m) * N + n) = s;
        else
          *reinterpret_cast<uint2*>(out + (uint64_t)m * N + n) = pack_bf16x4(s);
      }
    }
  }
