// Statements of the decode kernel (described in gemm_skinny.h), included in the body of
// gemm_decode_kernel and of gemm_decode_body, as gemm_skinny_body.h is and for its
// reason.  Uses the function's parameters and `epi`; no include guard.
  constexpr int NT = 2;  // 16-column MFMA tiles of the range (R <= 32)
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t w = blockIdx.x;
  const uint32_t c0 = 4 * (w * units_base + min(w, units_rem));
  const uint32_t R = 4 * (units_base + (w < units_rem ? 1u : 0u));  // columns = weight rows
  const uint32_t G = K / kGroup, rowb = K + 16;
  const uint32_t l16 = lane & 15, q = lane >> 4;

  // this wave's activation fragments and scales (L2-resident: every
  // workgroup reads them), and weight scales: issued first, ahead of the
  // weight stream.  Slot j holds
  // block wave + 8*((j + w) mod GW): the workgroups start their activation
  // reads at different blocks, so that the 32 CUs of an XCD do not all ask
  // its L2 for the same lines at once.
  const uint32_t nb_last = N / kGroup - 1, rot = w % GW;
  auto blk = [&](int j) __attribute__((always_inline)) -> uint32_t {
    const uint32_t jr = (uint32_t)j + rot;
    return wave + 8 * (jr >= (uint32_t)GW ? jr - GW : jr);
  };
  const __amdgpu_buffer_rsrc_t rA = make_rsrc(A, M * K);  // M * K < 2^31 here
  v8i af[GW][TM];
  float as[GW][TM], ws[GW][NT];
#pragma unroll
  for (int j = 0; j < GW; ++j) {
    const uint32_t b = min(blk(j), G - 1);  // blocks past G: loaded, not used
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      // rows past M read at an offset beyond the buffer's range, which gives
      // zeros without a memory request (not a load under a branch: that
      // load would be waited for inside the branch, one L2 round trip per
      // fragment)
      const uint32_t m = 16 * tm + l16;
      const uint32_t off = m < M ? m * K + b * kGroup + 32 * q : 0x80000000u;
      af[j][tm] = join(__builtin_amdgcn_raw_buffer_load_b128(rA, off, 0, 0),
                       __builtin_amdgcn_raw_buffer_load_b128(rA, off + 16, 0, 0));
      as[j][tm] = As[(uint64_t)b * Mp + min(m, Mp - 1)];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
      ws[j][t] = ROW ? 1.0f : Ws[min((c0 + 16 * t + 4 * q) / kGroup, nb_last) * G + b];
  }
  // the weight rows: piece p of row r is bytes [1024 p, 1024 p + 1024) (the
  // last piece of a row may be shorter); loads dealt round robin to the waves
  const __amdgpu_buffer_rsrc_t rW = make_rsrc(W + (uint64_t)c0 * K, R * K);
  const uint32_t pieces = (K + 1023) / 1024, lds0 = lds_addr(smem);
#pragma unroll 1
  for (uint32_t i = wave; i < R * pieces; i += 8) {
    const uint32_t r = i / pieces, p = i % pieces;
    if (1024 * p + 16 * lane < K) dma16_at(rW, r * K + 1024 * p + 16 * lane, 0, lds0 + r * rowb + 1024 * p);
  }
  // the loaded registers are pinned here, before the wait: the compiler
  // would otherwise sink loads into the compute branches below, after the
  // barrier, and pay a second memory round trip there
#pragma unroll
  for (int j = 0; j < GW; ++j) {
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)  // (16-byte operands: valid on the host pass too)
      asm volatile("" ::"v"(af[j][tm].lo), "v"(af[j][tm].hi), "v"(as[j][tm]));
#pragma unroll
    for (int t = 0; t < NT; ++t) asm volatile("" ::"v"(ws[j][t]));
  }
  wait_vmcnt<0>();
  wg_barrier();

  // all weight fragments of this wave's blocks, then the products, then the
  // promotions (no LDS or MFMA latency between dependent steps); blocks past
  // G and rows past R give zero fragments
  v8i wf[GW][NT];
#pragma unroll
  for (int j = 0; j < GW; ++j)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t r = 16 * t + l16, b = min(blk(j), G - 1);
      const uint8_t* wr = smem + min(r, R - 1) * rowb + b * kGroup + 32 * q;
      wf[j][t] = join(*reinterpret_cast<const u32x4*>(wr), *reinterpret_cast<const u32x4*>(wr + 16));
      if (r >= R || blk(j) >= G) wf[j][t] = v8i{0, 0, 0, 0, 0, 0, 0, 0};
    }
  v4f acc[NT][TM];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      v4f p[GW];
#pragma unroll
      for (int j = 0; j < GW; ++j) p[j] = mfma_e4m3_128(wf[j][t], af[j][tm]);
      acc[t][tm] = p[0] * (as[0][tm] * ws[0][t]);
#pragma unroll
      for (int j = 1; j < GW; ++j) acc[t][tm] += p[j] * (as[j][tm] * ws[j][t]);
    }
  wait_lgkm0();  // this wave's reads of the weight rows (s_barrier alone waits for none)
  wg_barrier();  // every wave done with the weight rows: LDS takes the partial tiles
  epi.template add_shared<TM, NT, 512>([&](int tm, int t) -> v4f& { return acc[t][tm]; }, smem, 0, c0, M, lane,
                                       wave, 8);
  v4f* red = reinterpret_cast<v4f*>(smem);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) red[((wave * NT + t) * TM + tm) * 64 + lane] = acc[t][tm];
  wait_lgkm0();
  wg_barrier();
  // waves share the final sums: wave v adds and stores tiles (t, tm) with
  // t*TM + tm = v (mod 8), the partials in wave order
  for (uint32_t jt = wave; jt < (uint32_t)(NT * TM); jt += 8) {
    const uint32_t t = jt / TM, tm = jt % TM;
    if (16 * t >= R) continue;
    v4f sum = red[(t * TM + tm) * 64 + lane];
    for (uint32_t v = 1; v < 8; ++v) sum += red[((v * NT + t) * TM + tm) * 64 + lane];
    const uint32_t m = 16 * tm + l16, n = c0 + 16 * t + 4 * q;
    if constexpr (ROW) {
      if (n < c0 + R) {
        const float4 rs = *reinterpret_cast<const float4*>(Ws + n);
        sum *= v4f{rs.x, rs.y, rs.z, rs.w};
      }
    }
    if (m < M && n < c0 + R) *reinterpret_cast<uint2*>(out + (uint64_t)m * N + n) = pack_bf16x4(sum);
  }
