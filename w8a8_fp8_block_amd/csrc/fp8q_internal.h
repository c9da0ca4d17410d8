// Internal launch interface between the C-ABI layer (fp8q_api.hip) and the
// kernel translation units.  Launchers assume validated arguments: shapes
// checked, pointers non-NULL and aligned, M > 0.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {

constexpr uint32_t kGroup = 128;  // K elements per scale group / weight block edge

// native 128-/64-bit vectors (usable with the nontemporal builtins)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// ---- quantizer geometry (shared with the selector) ----
// Variant A: flat over all M*(K/128) groups, 8 lanes per group,
// kQuantAWaves waves per workgroup.
constexpr uint32_t kQuantAWaves = 4;
constexpr uint32_t kQuantAGroupsPerWg = 8 * kQuantAWaves;
// Its form with the K-major scales beyond kQuantTileMinGroups groups:
// workgroups of kQuantTileRows waves, each covering kQuantTileRows token
// rows x kQuantTileGroups groups (wave v: row v of the tile, one group per 8
// lanes).  Up to that many groups the flat order writes the K-major scales
// itself (back to back: 2.55-3.02 us at M = 16 / 25 against 2.55-3.18 for
// the tiles, 5.31 / 6.41 against 5.57 / 6.94 at M = 1168, K = 5120 / 6144).
constexpr uint32_t kQuantTileRows = 8, kQuantTileGroups = 8;
constexpr uint64_t kQuantTileMinGroups = 1u << 17;
// Variant B: K-grouped; a workgroup covers kQuantBGroupsPerWg consecutive
// groups of one token row, kQuantBRounds groups per 16-lane row.
constexpr uint32_t kQuantBWaves = 4;
constexpr uint32_t kQuantBRounds = 2;
constexpr uint32_t kQuantBGroupsPerWg = 4 * kQuantBWaves * kQuantBRounds;
// Floor of the selection rule (workgroups per CU variant B's grid must
// reach before it may run).  The value is the page's: on gfx950 there is no
// crossover to derive another one from.  Timed by kernel duration over the
// 30 shapes of the token/K sweep (M in 16..16384, K in 5120/6144/17408, cold
// input), B was never faster than A by more than 0.1 us, and it was 12-33%
// slower from M = 4576 on, where its grid (9152-81920 workgroups on 256 CUs)
// fills the device many times over.  The floor only matters where B is
// requested.
constexpr uint32_t kQuantMinWgPerCu = 2;
// Target default of the lever that lets variant B run at all: off on gfx950,
// for the measurements above (FP8Q_QUANT_VARIANT=floor requests B, "b"
// forces it).
constexpr bool kQuantBRequestedByDefault = false;

// Quantizer variants A and B: codes q [M,K], row-major scales scale_rm
// [M,K/128] (may be NULL) and, when scale_km is not NULL, the K-major scales
// [K/128, ceil16(M)] as well; the groups of the last token row then also
// write +0.0 to the pad slots M .. ceil16(M)-1 of their column.
hipError_t launch_quant_a(const uint16_t* x, uint8_t* q, float* scale_rm,
                          float* scale_km, uint32_t M, uint32_t K, hipStream_t s);
hipError_t launch_quant_b(const uint16_t* x, uint8_t* q, float* scale_rm,
                          float* scale_km, uint32_t M, uint32_t K, hipStream_t s);

hipError_t launch_relayout(const float* scale_rm, float* scale_km, uint32_t M,
                           uint32_t K, hipStream_t s);

// GEMM kernels: LDS-tiled MFMA (tile configuration cfg: 0/1 = 128x128
// tiles, 4 waves, 2 LDS stages so that two workgroups share a CU; 2 =
// 256x128 with 8 waves; 3 = 256x128 with 4 waves; 4 = 256x128 with two
// ping-pong groups of 4 waves) and skinny (M <= 64).
constexpr uint32_t kSkinnyMaxM = 65535u * 64u;  // skinny kernel: row tiles of 64 (grid y <= 65535)
// row_scaled: w_s is one fp32 scale per weight row [N] (applied to the
// finished accumulator) instead of [N/128, K/128] block scales.
hipError_t launch_gemm_tiled(const uint8_t* a, const float* a_s_km, const uint8_t* w,
                             const float* w_s, uint16_t* out, uint32_t M, uint32_t N,
                             uint32_t K, int cfg, bool row_scaled, hipStream_t s);
// Split-K form of the 128x128 tiled kernel (block-scaled weights): splits
// workgroups per tile, each over a contiguous range of K blocks, write fp32
// partial tiles to part [splits, M, N]; a reduction adds them in split order
// into out.  2 <= splits <= K/128; cus = the device's compute units (a grid
// of at most one workgroup per CU takes the three-stage form).
hipError_t launch_splitk_128(const uint8_t* a, const float* a_s_km, const uint8_t* w,
                             const float* w_s, uint16_t* out, float* part, uint32_t M,
                             uint32_t N, uint32_t K, uint32_t splits, uint32_t cus,
                             hipStream_t s);
// The reduction alone: out = bf16(sum of part [splits, M, N] in split order).
hipError_t launch_splitk_reduce(const float* part, uint16_t* out, uint32_t M, uint32_t N,
                                uint32_t splits, hipStream_t s);
// Stream-K form of the 256x128 ping-pong kernel (block-scaled weights): cus
// persistent workgroups (a multiple of 8, at most the device's CUs); whole
// tiles in data-parallel rounds, the last partial round's tiles cut along K
// into pieces for the otherwise idle workgroups, the pieces summed through
// fp32 partials and per-wave flags in the caller's workspace of
// gemm_streamk_workspace_bytes(cus) bytes (contents on entry ignored).
// gemm_streamk_applies: whether a plan exists for the shape and, unless
// forced, is predicted at least 10% shorter than the data-parallel kernel.
bool gemm_streamk_applies(uint32_t M, uint32_t N, uint32_t K, uint32_t cus, bool forced);
uint64_t gemm_streamk_workspace_bytes(uint32_t cus);
hipError_t launch_gemm_streamk(const uint8_t* a, const float* a_s_km, const uint8_t* w,
                               const float* w_s, uint16_t* out, void* workspace, uint32_t M,
                               uint32_t N, uint32_t K, uint32_t cus, bool forced, hipStream_t s);
// Split-K form of the skinny kernel for M <= 64 (block-scaled weights): the
// partials of `splits` K ranges in part [splits, M, N], then the ordered
// reduction into out.  False, with nothing launched, where M > 64 or the
// column ranges of cus / splits workgroups would exceed 128 columns.
bool launch_skinny_split(const uint8_t* a, const float* a_s_km, const uint8_t* w,
                         const float* w_s, uint16_t* out, float* part, uint32_t M, uint32_t N,
                         uint32_t K, uint32_t splits, uint32_t cus, hipStream_t s,
                         hipError_t& err);
// Whether the skinny path runs the decode kernel (the whole weight slice of
// a workgroup in LDS) for this shape.
bool decode_takes(uint32_t M, uint32_t N, uint32_t K, uint32_t cu_count);
// Workgroups per split and columns a workgroup owns at most in the skinny
// kernel's split form with `splits` K ranges on `cus` compute units.
uint32_t skinny_split_grid(uint32_t N, uint32_t splits, uint32_t cus);
uint32_t skinny_split_columns(uint32_t N, uint32_t splits, uint32_t cus);
hipError_t launch_gemm_skinny(const uint8_t* a, const float* a_s_km, const uint8_t* w,
                              const float* w_s, uint16_t* out, uint32_t M, uint32_t N,
                              uint32_t K, uint32_t cu_count, bool row_scaled, hipStream_t s);
// Name (with template arguments) of the kernel launch_gemm_skinny runs for
// this shape: the decode kernel or the fragment-layout skinny kernel.
void gemm_skinny_kernel_name(uint32_t M, uint32_t N, uint32_t K, uint32_t cu_count,
                             bool row_scaled, char* buf, size_t len);

// bf16 comparator GEMM: out[M,N] = bf16(x[M,K] . w[N,K]^T), N % 128 == 0,
// K % 64 == 0.
hipError_t launch_gemm_bf16(const uint16_t* x, const uint16_t* w, uint16_t* out, uint32_t M,
                            uint32_t N, uint32_t K, hipStream_t s);

// FP8 weights [N,K] -> bf16 [N,K]: dst = bf16(fl32(dec(w) * scale[(n/bn)*sk + k/bk]))
// with (bn, bk, sk) = (128, 128, K/128) or, per_row, (1, K, 1).
hipError_t launch_dequant(const uint8_t* w, const float* scale, uint16_t* dst, uint32_t N,
                          uint32_t K, bool per_row, hipStream_t s);

// FFN intermediate: h = bf16(silu(gate) * up) for bf16 gate/up [M,I], then
// quantized per (token, 128-group): codes [M,I] and K-major scales
// [I/128, ceil16(M)] with the pad slots zeroed.
hipError_t launch_silu_mul_quant(const uint16_t* gate, const uint16_t* up, uint8_t* q,
                                 float* scale_km, uint32_t M, uint32_t I, hipStream_t s);

// Fused gate/up projection of the dense FFN: x codes [M,H] with K-major
// scales [H/128, ceil16(M)], gate and up weights [I,H] with block scales
// [I/128, H/128] -> the intermediate's codes [M,I] and K-major scales
// [I/128, ceil16(M)] (pad slots zeroed), equal to launch_silu_mul_quant of
// the two bf16 projections.  I % 128 == 0, H % 128 == 0.
hipError_t launch_ffn_gate_up(const uint8_t* x, const float* x_s_km, const uint8_t* w_gate,
                              const float* ws_gate, const uint8_t* w_up, const float* ws_up,
                              uint8_t* hq, float* hs_km, uint32_t M, uint32_t H, uint32_t I,
                              hipStream_t s);

// ---- expert routing (route.hip) ----
constexpr uint32_t kMaxExperts = 512, kMaxTopK = 32;
// Top-k choice of each token with softmax weights, and the grouping of the
// slots t * top_k + j by expert: order (stable; slots without an expert last),
// pos (its inverse), offsets [E + 1].  workspace: route_workspace_bytes.
uint64_t route_workspace_bytes(uint32_t T, uint32_t E);
hipError_t launch_route(const void* logits, bool bf16, int32_t* ids, float* weights, int32_t* order,
                        int32_t* pos, int32_t* offsets, void* workspace, uint32_t T, uint32_t E,
                        uint32_t top_k, bool renorm, hipStream_t s);
// The grouping alone, of n given ids (outside 0 .. groups-1: no group).
uint64_t group_workspace_bytes(uint32_t n, uint32_t groups);
hipError_t launch_group_rows(const int32_t* ids, int32_t* order, int32_t* pos, int32_t* offsets,
                             void* workspace, uint32_t n, uint32_t groups, hipStream_t s);
// out[t] = bf16(sum_j weights[t][j] * y[pos[t][j]]), H % 8 == 0.
hipError_t launch_combine(const uint16_t* y, const float* weights, const int32_t* pos,
                          const int32_t* offsets, uint16_t* out, uint32_t T, uint32_t E,
                          uint32_t top_k, uint32_t H, hipStream_t s);

// ---- products grouped by expert (grouped.hip) ----
// Sorted rows p of expert e (offsets[e] <= p < offsets[e + 1]) read activation
// row order[p] / per_row (order NULL: row p) of a_rows; weights w [E, N, K]
// with block scales [E, N/128, K/128]; out [R, N].  Kernel ids: 1 weight
// streaming, 2 128 x 128 tiles, 3 persistent ping-pong 128 x 256 tiles; group_gemm_auto
// picks by the mean rows an expert and the number of tiles.
int group_gemm_auto(uint32_t R, uint32_t E, uint32_t N, uint32_t cus);
hipError_t launch_gemm_grouped(const uint8_t* a, const float* a_s_km, const uint8_t* w,
                               const float* w_s, uint16_t* out, const int32_t* offsets,
                               const int32_t* order, uint32_t per_row, uint32_t a_rows, uint32_t R,
                               uint32_t E, uint32_t N, uint32_t K, uint32_t cus, int kernel,
                               hipStream_t s);
// Gate and up of the same rows in one launch, bf16 out [R, I] each.
hipError_t launch_group_gate_and_up(const uint8_t* x, const float* x_s_km, const uint8_t* w_gate,
                                    const float* ws_gate, const uint8_t* w_up, const float* ws_up,
                                    uint16_t* gate, uint16_t* up, const int32_t* offsets,
                                    const int32_t* order, uint32_t per_row, uint32_t a_rows, uint32_t R,
                                    uint32_t E, uint32_t H, uint32_t I, uint32_t cus, int kernel,
                                    hipStream_t s);
// Gate, up, SiLU and requantization in one kernel: codes hq [R, I] and K-major
// scales hs_km [I/128, ceil16(R)] (rows of no expert are left as they are).
hipError_t launch_group_ffn_gate_up(const uint8_t* x, const float* x_s_km, const uint8_t* w_gate,
                                    const float* ws_gate, const uint8_t* w_up, const float* ws_up,
                                    uint8_t* hq, float* hs_km, const int32_t* offsets,
                                    const int32_t* order, uint32_t per_row, uint32_t a_rows, uint32_t R,
                                    uint32_t E, uint32_t H, uint32_t I, uint32_t cus, hipStream_t s);

// ---- low-rank adapters beside the projection (lora.hip) ----
constexpr uint32_t kMaxLoraRank = 128;
// One pass over x: its codes and scales (both layouts, pad slots zeroed), and
// v = x . A^T of the rows with an adapter into workspace (lora_workspace_bytes).
uint64_t lora_workspace_bytes(uint32_t M, uint32_t K, uint32_t rank);
hipError_t launch_lora_quant_shrink(const uint16_t* x, const uint16_t* a, const int32_t* ids, uint8_t* x_q,
                                    float* x_s_rm, float* x_s_km, void* workspace, uint32_t M, uint32_t K,
                                    uint32_t adapters, uint32_t rank, hipStream_t s);
// The block-scaled GEMM (kernel ids of launch_gemm: 1, 2 or 5; splits >= 2:
// its split form with part [splits, M, N]) plus scale * v . B^T.
hipError_t launch_lora_gemm(const uint8_t* a, const float* a_s_km, const uint8_t* w, const float* w_s,
                            uint16_t* out, const void* workspace, float* part, const uint16_t* lora_b,
                            const float* lora_scale, const int32_t* ids, uint32_t M, uint32_t N, uint32_t K,
                            uint32_t adapters, uint32_t rank, uint32_t cus, int kernel, uint32_t splits,
                            hipStream_t s);

// ---- a training step through the projection ----
// RMS norm (norm.hip): h = bf16(x + r) (r NULL: h = x, h unused), codes q of
// h * rstd * w with their scales in either layout, bf16 y and rstd where not NULL.
constexpr uint32_t kMaxNormK = 32768;
hipError_t launch_norm_quant(const uint16_t* x, const uint16_t* r, const uint16_t* w, uint16_t* h, uint16_t* y,
                             uint8_t* q, float* scale_rm, float* scale_km, float* rstd, float eps, uint32_t M,
                             uint32_t K, hipStream_t s);
// Its gradient: dx = dh + d(norm) (dh NULL: none), dw [K] fp32; M = 0: dw = 0.
uint64_t norm_grad_workspace_bytes(uint32_t M, uint32_t K);
hipError_t launch_norm_grad(const uint16_t* dy, const uint16_t* dh, const uint16_t* h, const uint16_t* w,
                            const float* rstd, uint16_t* dx, float* dw, void* workspace, uint32_t M, uint32_t K,
                            hipStream_t s);
// Row codes with K-major scales (q NULL: not wanted) and token codes with their
// exponent bytes [ceil(M/512), K, 4] (quant_dual.hip).
hipError_t launch_quant_dual(const uint16_t* x, uint8_t* q, float* scale_km, uint8_t* q_tok, uint8_t* exp_tok,
                             uint32_t M, uint32_t K, hipStream_t s);
// Gradients of the block-scaled product (dgrad.hip, wgrad.hip): dx [M,K] from row codes dy
// [M,N] and w [N,K]; dw [N,K] from token codes dy [M,N] and x [M,K].  splits >= 2: the sum
// cut into as many ranges, their fp32 results in part.  wide: dx in tiles of 256 rows, not 128.
hipError_t launch_gemm_dgrad(const uint8_t* dy, const float* dy_s_km, const uint8_t* w, const float* w_s, uint16_t* dx,
                             float* part, uint32_t M, uint32_t N, uint32_t K, bool wide, uint32_t splits,
                             hipStream_t s);
hipError_t launch_gemm_wgrad(const uint8_t* dy, const uint8_t* ey, const uint8_t* x, const uint8_t* ex, uint16_t* dw,
                             float* part, uint32_t M, uint32_t N, uint32_t K, uint32_t splits, uint32_t cus,
                             hipStream_t s);
// Balance loss of a router and the gradient of its logits (balance.hip).
uint64_t balance_workspace_bytes(uint32_t T, uint32_t E);
hipError_t launch_balance(const void* logits, bool bf16, const int32_t* ids, int32_t* counts, float* prob, float* loss,
                          void* workspace, float coef, uint32_t T, uint32_t E, uint32_t top_k, hipStream_t s);
hipError_t launch_route_grad(const void* logits, bool bf16, const int32_t* ids, const float* dweights,
                             const int32_t* counts, const float* dloss, void* dlogits, float coef, uint32_t T,
                             uint32_t E, uint32_t top_k, bool renorm, hipStream_t s);

// Clock stamps (measurement support): n one-wave workgroups each write
// {XCD id, HW_ID, shader clock counter, 100 MHz counter} to dst[4*i .. 4*i+3].
hipError_t launch_clock_stamp(unsigned long long* dst, uint32_t n, hipStream_t s);

inline uint32_t m_pad16(uint32_t m) { return (m + 15u) / 16u * 16u; }

}  // namespace fp8q
