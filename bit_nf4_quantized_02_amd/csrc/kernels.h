// Internal launch functions of libqlora (host side). Each enqueues kernels on
// `stream` and returns hipGetLastError(); argument checking happens before,
// in api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qlora.h"

namespace qlora {

inline size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

// ---- encoder workspace: absmax fp32 [nb], run sums fp64 [ceil(nb/256)]
inline size_t quantize_ws_absmax_bytes(int64_t nb) { return align256((size_t)nb * 4); }
inline size_t quantize_ws_runsum_bytes(int64_t nb) { return align256((size_t)((nb + 255) / 256) * 8); }
inline size_t quantize_ws_bytes(int64_t nb) {
  return quantize_ws_absmax_bytes(nb) + quantize_ws_runsum_bytes(nb) + align256((size_t)((nb + 255) / 256) * 4);
}

// code8 NULL: no double quantization, s2 receives one scale per block, fp32
// or (s2_bf16) the bf16 rounding of the block absmax, which the codes are
// then taken against.
hipError_t launch_quantize(const void* W, bool w_bf16, int64_t n, int64_t k, const float* codebook,
                           uint8_t* codes, uint8_t* code8, float* s2, float* mean, void* ws,
                           hipStream_t stream, bool s2_bf16 = false);

// Encoded weight as the kernels see it (s2_bf16: without double
// quantization, s2 holds bf16 bit patterns, one per block).
struct Nf4View {
  int64_t n, k;
  const uint8_t* codes;
  const uint8_t* code8;
  const float* s2;
  const float* mean;
  const float* codebook;
  bool s2_bf16 = false;
};

hipError_t launch_dequant(const Nf4View& w, uint16_t* out, hipStream_t stream, bool f16 = false);

// Columns of the LoRA "extra" contraction region: [hi | lo] halves of the
// scaled low-rank activation, padded with zeros to a multiple of 64.
inline int lora_extra_cols(int r) { return r > 0 ? ((2 * r + 63) / 64) * 64 : 0; }

// out[m, j] = sum_c P[m, c] Q(c, j), P bf16 [M, C]; Q bf16 [r, C] (q_layout
// 0) or [C, r] (q_layout 1); fp32 out [M, r] (nullable). If split != NULL it
// also receives rows [bf16(scale*out) | bf16(scale*out - hi) | 0 ...] of
// lora_extra_cols(r) elements. part: workspace of rowdot_ws_bytes (may be 0).
size_t rowdot_ws_bytes(int64_t M, int64_t C, int r);
// pmask (uint8 [M, C], q_layout 0 and C % 8 == 0 only; NULL: none): P's
// elements whose byte is 0 read as zero (dropout on the adapter's input).
hipError_t launch_rowdot(const uint16_t* P, int64_t M, int64_t C, const uint16_t* Q, int q_layout, int r,
                         float* out, uint16_t* split, float scale, float* part, hipStream_t stream,
                         const uint8_t* pmask = nullptr, bool f16 = false);

// out / split (as launch_rowdot's) from partials [ns][M][r], added in order.
hipError_t launch_rowdot_finalize(const float* part, int ns, int64_t M, int r, float* out, uint16_t* split, float scale,
                                  hipStream_t stream, bool f16);

// Column reduction over M in fixed order, for the adapter gradients:
//   G[c, j] (+)= scale * sum_m P[m, c] * Q[m, j]    P bf16 [M, C], Q fp32 [M, r]
// written at G[c * g_sc + j * g_sj]. partial (fp32, [splits, C, r]) is workspace.
size_t coldot_ws_bytes(int64_t M, int64_t C, int r);
hipError_t launch_coldot(const uint16_t* P, int64_t M, int64_t C, const float* Q, int r, float scale,
                         float* G, int64_t g_sc, int64_t g_sj, int accumulate, float* partial,
                         hipStream_t stream, const uint8_t* pmask = nullptr, bool f16 = false);
// dA and dB of one layer in one launch (both with a single token split, no
// mask): products (P0, C0, Q0 -> G0 with strides g_sc0, g_sj0) and (P1, ...),
// the same arithmetic as two launch_coldot calls. coldot_pairable tells when
// it applies.
bool coldot_pairable(int64_t M, int64_t C0, int64_t C1);
hipError_t launch_coldot_pair(const uint16_t* P0, int64_t C0, const float* Q0, float* G0, int64_t g_sc0,
                              int64_t g_sj0, const uint16_t* P1, int64_t C1, const float* Q1, float* G1,
                              int64_t g_sc1, int64_t g_sj1, int64_t M, int r, float scale, int accumulate,
                              hipStream_t stream, bool f16);

// Y = RN_bf16(X W'^T + [sT_hi | sT_lo] [B | B]^T): fused dequant + MFMA GEMM.
hipError_t launch_gemm_fwd(const Nf4View& w, const uint16_t* X, int64_t M, const uint16_t* TS,
                           const uint16_t* B, int r, uint16_t* Y, hipStream_t stream);

// dX = RN_bf16(dY W' + [sU_hi | sU_lo] [A ; A]): fused transposed dequant + MFMA GEMM.
hipError_t launch_gemm_dx(const Nf4View& w, const uint16_t* dY, int64_t M, const uint16_t* US,
                          const uint16_t* A, int r, uint16_t* dX, hipStream_t stream,
                          const uint8_t* mask = nullptr, float keep_scale = 1.0f);

// dX = RN_bf16(dY W + [sU_hi | sU_lo] [A ; A]) for a bf16 base weight W [n, k]
// (k % 64 == 0): the fused kernel's dX with the weight tile copied instead of
// expanded.
hipError_t launch_gemm_w16_dx(const uint16_t* W, int64_t n, int64_t k, const uint16_t* dY, int64_t M,
                              const uint16_t* US, const uint16_t* A, int r, uint16_t* dX, hipStream_t stream);

// Expanded bf16 operand of the plain GEMM (forward [n, k + xc], or dX
// [k, np + xc] with np = n rounded up to 64), LoRA factor appended.
int64_t expand_pad_rows(int64_t n);
size_t expand_ws_bytes(int64_t n, int64_t k, int r, bool transposed);
hipError_t launch_expand(const Nf4View& w, const uint16_t* lr, int r, bool transposed, uint16_t* out,
                         hipStream_t stream, bool f16 = false);
// The dX operand in contraction-major form for the GEMM's NN form (n % 64
// == 0): out [n + xc, k], rows 0 .. n-1 W' as the forward expansion writes
// them, then the low-rank rows [A ; A ; 0].
size_t expand_nn_bytes(int64_t n, int64_t k, int r);
hipError_t launch_expand_nn(const Nf4View& w, const uint16_t* A, int r, uint16_t* out, hipStream_t stream);

// [n, lora_extra_cols(r)] rows [B | B | 0] (bf16), the low-rank operand of
// the forward GEMM when the weight operand is a separate matrix.
hipError_t launch_lowrank_rows(const uint16_t* B, int64_t n, int r, uint16_t* out, hipStream_t stream);

// out = RN_bf16([act | split] F^T) over an expanded operand F [nout, kcp + kx].
// The kernel addresses each operand with 32-bit byte offsets: every operand
// must be smaller than 4 GiB (gemm_bf16_offsets_fit). When the last wave of
// 256 tiles holds at most 128 (all of them, for small outputs), those tiles
// are split along the contraction over gemm_bf16_splits() workgroups each,
// whose fp32 partials (gemm_bf16_ws_bytes() of workspace, `part`) are added
// in split order and rounded once; part may be NULL when that size is 0.
bool gemm_bf16_offsets_fit(int64_t M, int64_t kc, int kx, int64_t nout);
int gemm_bf16_splits(int64_t M, int64_t kc, int kx, int64_t nout);
size_t gemm_bf16_ws_bytes(int64_t M, int64_t kc, int kx, int64_t nout);
// How a 256 x 256-tile GEMM of nk steps spreads its tiles: the first `full`
// whole, the `tail` after them split `splits` ways along the contraction.
struct GemmSplit {
  int64_t full, tail;
  int splits;
};
GemmSplit gemm_split_plan(int64_t M, int64_t nout, int64_t nk);
// Tail tiles' partials [splits][tail][256 x 256], added in split order and rounded once.
hipError_t launch_gemm_reduce(const float* part, const GemmSplit& sp, int64_t M, int64_t nout, uint16_t* out,
                              hipStream_t stream, bool f16);
// mask (uint8 [M, nout], may be NULL): dropout on the low-rank term, which is
// multiplied by keep_scale where mask is set and dropped where it is not,
// before the main contraction is added (one rounding of the whole sum).
hipError_t launch_gemm_bf16(const uint16_t* act, int64_t M, int64_t kc, const uint16_t* split, int kx,
                            const uint16_t* f, int64_t nout, uint16_t* out, float* part, hipStream_t stream,
                            const uint8_t* mask = nullptr, float keep_scale = 1.0f, bool f16 = false);

// The same GEMM with the weight operand and the low-rank operand as separate
// row-major matrices: f [nout, ldf] (the base contraction in its first kc
// columns; kc % 64 == 0 or the columns up to the next multiple of 64 zero)
// and fx [nout, ldx] (kx low-rank columns). A bf16 base weight W [n, k] is
// such an f for the forward as it is stored.
// nn: f is stored [contraction][output] instead ([kc rows, ldf], kc % 64 == 0,
// and fx [kx rows, ldx]): dX over a bf16 base weight W [n, k] as stored, the
// fragments read through the transposing LDS read (bf16, no mask).
hipError_t launch_gemm_bf16_ext(const uint16_t* act, int64_t M, int64_t kc, const uint16_t* split, int kx,
                                const uint16_t* f, int64_t ldf, const uint16_t* fx, int64_t ldx, int64_t nout,
                                uint16_t* out, float* part, hipStream_t stream, const uint8_t* mask = nullptr,
                                float keep_scale = 1.0f, bool f16 = false, bool nn = false,
                                const float* row_scale = nullptr);

// Ranks padded to what the kernels that take factors in operand order are built for.
inline int rank_pad(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }
// A factor (layout 0: [r, C], 1: [C, r]) in operand order [Cp / 32][rank_pad(r)
// / 16][64 lanes][16 bytes], zero past C (Cp: a multiple of 32); Q1's (not NULL)
// after it.
size_t operand_order_bytes(int64_t Cp, int r);
// split16: Q is fp16 and given as two bf16 parts, one after the other for each
// 32 columns (twice the bytes).
hipError_t launch_operand_order(const uint16_t* Q, const uint16_t* Q1, int layout, int64_t C, int64_t Cp, int r,
                                uint16_t* out, hipStream_t stream, bool split16 = false);

// One factor Q in operand order as above and the other as low-rank operand rows
// [nf, lora_extra_cols(r)]: layout 0 (forward) Q = A [r, C], F = B [nf, r], rows
// [B | B | 0]; 1 (dX) Q = B [C, r], F = A [r, nf], row c = [A[:, c] | A[:, c] | 0].
hipError_t launch_factors(const uint16_t* Q, int layout, int64_t C, int64_t Cp, int r, uint16_t* order,
                          const uint16_t* F, int64_t nf, uint16_t* rows, hipStream_t stream);

// [lora_extra_cols(r), k] rows [A ; A ; 0] (bf16), the low-rank operand of the
// nn GEMM (dX over a bf16 base).
hipError_t launch_lowrank_cols(const uint16_t* A, int r, int64_t k, uint16_t* out, hipStream_t stream);

// Adapter merge: out = round(W' + scale * B A) (w != NULL; bf16, or fp32 if
// out_f32) or unmerge: out = RN_bf16(Wm - scale * B A) (w == NULL, Wm bf16).
size_t merge_smem_bytes(int r);
hipError_t launch_merge(const Nf4View* w, const uint16_t* Wm, int64_t n, int64_t k, const uint16_t* A,
                        const uint16_t* B, int r, float scale, bool out_f32, void* out, hipStream_t stream);

// Small-M dequant-GEMV: Y = RN_bf16(X W'^T + scale * T B^T), M <= 16. ws:
// gemv_ws_bytes(k) bytes for the activations in operand order.
size_t gemv_ws_bytes(int64_t k);
// The GEMV addresses the codes with 32-bit buffer offsets: n k / 2 bytes
// (plus one workgroup's rows past n) under 4 GiB.
bool gemv_fits(int64_t n, int64_t k);
hipError_t launch_gemv(const Nf4View& w, const uint16_t* X, int64_t M, const float* T,
                       const uint16_t* B, int r, float scale, uint16_t* Y, void* ws, hipStream_t stream,
                       bool f16 = false);

// The layer forward behind qlora_linear_fwd and its dropout / fp16 forms
// (api.hip), and the workspace it carves for a bf16 call with or without a
// caller-provided T_save.
qlora_status linear_fwd_impl(const qlora_nf4_weight* w, const void* X, int64_t M, const void* A, const void* B,
                             int r, float scale, const uint8_t* mask, float keep_scale, void* Y, float* T_save,
                             void* ws, size_t ws_bytes, void* stream, bool f16 = false);
size_t linear_fwd_ws_bytes(int64_t M, int64_t n, int64_t k, int r, bool have_tsave);

// Small-M dX through the frozen base (M <= 16): dX = RN_bf16(dY W' + scale
// (U A) [. mask * keep]) with U = dY B fp32 [M, r] (nullable when r == 0)
// and A bf16 [r, k]; ws: gemv_dx_ws_bytes(n, k) bytes of fp32 partials.
size_t gemv_dx_ws_bytes(int64_t n, int64_t k);
hipError_t launch_gemv_dx(const Nf4View& w, const uint16_t* dY, int64_t M, const float* U, const uint16_t* A, int r,
                          float scale, uint16_t* dX, void* ws, hipStream_t stream, const uint8_t* mask = nullptr,
                          float keep = 1.0f);

// ---- adapter gradients of the feed-forward operators (colgrad.hip)
// Q0 fp32 [W0][M][r], Q1 [W1][M][r] as bf16 parts in operand order (W 0: none).
size_t rank_parts_bytes(int64_t M, int r, int W);
hipError_t launch_rank_parts(const float* Q0, int W0, void* out0, const float* Q1, int W1, void* out1, int64_t M, int r,
                             hipStream_t stream);
// Gradients left as partials [splits][W][count], to be added in order (G1: w =
// 1; NULL: left out); W 0: none.
struct GradJob {
  const float* part;
  int64_t count;
  int splits, W;
  float *G0, *G1;
};
hipError_t launch_grad_reduce(const GradJob& a, const GradJob& b, float scale, int accumulate, hipStream_t stream);
// Gw (+)= scale P^T Qw from Q's parts, as [r, C] (j_first; C % 8 == 0, W 1 or
// 2) or [C, r] (W = 1); `job` is what launch_grad_reduce has to finish.
size_t colgrad_ws_bytes(int64_t M, int64_t C, int r, int W);
hipError_t launch_colgrad(const uint16_t* P, int64_t M, int64_t C, const void* parts, int W, int r, float scale,
                          float* G0, float* G1, bool j_first, int accumulate, float* part, GradJob& job,
                          hipStream_t stream, bool f16);

// ---- the gated feed-forward block H = silu(G) U over two NF4 weights
// Few tokens (M <= 16). G, U and T_save ([2][M][r]) may be NULL.
size_t gemv_pair_ws_bytes(int64_t M, int64_t n, int64_t k, int r);
hipError_t launch_gemv_pair(const Nf4View& g, const Nf4View& u, const uint16_t* X, int64_t M, const uint16_t* Ag,
                            const uint16_t* Bg, const uint16_t* Au, const uint16_t* Bu, int r, float scale, uint16_t* H,
                            uint16_t* G, uint16_t* U, float* T_save, void* ws, hipStream_t stream, bool f16);
// Low-rank columns of the block's GEMMs, [hi_g | lo_g | hi_u | lo_u | 0] of s T
// or s P (fp16: times 2^-e, by row).
inline int gated_extra_cols(int r) { return r > 0 ? ((4 * r + 63) / 64) * 64 : 0; }
// fp16: low-rank columns from partials [splits][W][M][r] added in order. out
// (NULL: not written) takes the sums [W][M][r]; split (NULL: not written) row m's
// columns [hi_0 | lo_0 | hi_1 | .. | 0] (xc in all) of scale * sums times 2^-e,
// and row_scale [row_scale_rows(M)] 2^e, with e so that the row's largest value
// lies in [2^14, 2^15): none leaves fp16's range, and lo's smallest step is 2^-39
// of it. apart: an e for each factor (row_scale [W][row_scale_rows(M)]), where
// their products are different outputs.
inline int64_t row_scale_rows(int64_t M) { return (M + 255) / 256 * 256; }  // whole tiles of rows
inline size_t row_scale_bytes(int64_t M, int W = 1) { return (size_t)row_scale_rows(M) * W * 4; }
hipError_t launch_scaled_columns(const float* part, int splits, int W, int64_t M, int r, int xc, float scale, float* out,
                                 uint16_t* split, float* row_scale, hipStream_t stream, bool apart = false);
// X Ag^T and X Au^T: T (NULL: not written) as [2][M][r], and the scaled
// columns in split (NULL: not written; fp16: with row_scale).
size_t gated_project_ws_bytes(int64_t M, int64_t k, int r);
hipError_t launch_gated_project(const uint16_t* X, int64_t M, int64_t k, const uint16_t* Ag, const uint16_t* Au, int r,
                                float scale, float* T, uint16_t* split, float* row_scale, void* ws, hipStream_t stream,
                                bool f16);
// Both weights expanded for the forward: rows in groups of 64, 32 gate rows
// then the same 32 up rows, [W' | low-rank columns], pitch k + extra.
inline int64_t gated_rows(int64_t n) { return (n + 31) / 32 * 64; }
size_t gated_fwd_operand_bytes(int64_t n, int64_t k, int r);
hipError_t launch_gated_expand_fwd(const Nf4View& g, const Nf4View& u, const uint16_t* Bg, const uint16_t* Bu, int r,
                                   uint16_t* out, hipStream_t stream, bool f16);
// The forward GEMM over it with the join in its epilogue (part as the plain
// GEMM's for gated_rows(n) outputs).
hipError_t launch_gemm_gated(const uint16_t* act, int64_t M, int64_t k, const uint16_t* split, int kx,
                             const float* row_scale, const uint16_t* f, int64_t n, uint16_t* H, uint16_t* G, uint16_t* U,
                             float* part, hipStream_t stream, bool f16);
// Both weights contraction-major for dX: [Wg ; 0 ; Wu ; 0 ; Ag ; Ag ; Au ; Au
// ; 0], each weight's rows padded to a multiple of 64, pitch k.
inline int64_t gated_pad(int64_t n) { return (n + 63) / 64 * 64; }
size_t gated_dx_operand_bytes(int64_t n, int64_t k, int r);
hipError_t launch_gated_expand_dx(const Nf4View& g, const Nf4View& u, const uint16_t* Ag, const uint16_t* Au, int r,
                                  uint16_t* out, hipStream_t stream, bool f16);
// D [M, 2 gated_pad(n)] = [dG | 0 | dU | 0] in 16 bits (D NULL: not written),
// and (r > 0) P = [dG Bg ; dU Bu] as fp32 [2][M][r] from the unrounded dG, dU,
// with its scaled hi / lo columns in split (NULL: not written; fp16: with row_scale).
size_t gated_join_ws_bytes(int64_t M, int64_t n, int r);
hipError_t launch_gated_join(const uint16_t* G, const uint16_t* U, const uint16_t* dH, int64_t M, int64_t n,
                             const uint16_t* Bg, const uint16_t* Bu, int r, float scale, uint16_t* D, float* P,
                             uint16_t* split, float* row_scale, void* ws, hipStream_t stream, bool f16);
// dBg = scale dG^T T[0], dBu = scale dU^T T[1] (either may be NULL) from T's
// parts, dG and dU unrounded; finished by launch_grad_reduce(job).
size_t gated_db_ws_bytes(int64_t M, int64_t n, int r);
hipError_t launch_gated_db(const uint16_t* G, const uint16_t* U, const uint16_t* dH, int64_t M, int64_t n,
                           const void* parts, int r, float* dBg, float* dBu, float* part, GradJob& job,
                           hipStream_t stream, bool f16);

// ---- the 8-bit layer (formats and layouts: fp8.h)
struct Fp8View {
  int64_t n, k;
  const uint8_t* codes;  // [n, k up to a multiple of 128]
  const uint8_t* scale;  // [ceil(n / 128), ceil(k / 128)]
};
hipError_t launch_fp8_encode(const void* W, int dt, int64_t n, int64_t k, uint8_t* codes, uint8_t* scale,
                             hipStream_t stream);
hipError_t launch_fp8_decode(const Fp8View& w, uint16_t* out, hipStream_t stream);
// Activations P [M, C] -> codes and scales ([M, C up to 128] and the GEMM's
// scale words; few: the GEMV's operand order in tiles of 16 rows, fp8_gemv_*_bytes),
// and for r > 0 the partials [splits][W][M][r] of P Q^T; W factors in operand
// order one after the other, for few one as it is, [r, C]. codes NULL (always
// for W = 2): the projections only. gcodes, gscale: P's codes and scales by row
// (qlora_fp8_rows), if it has them; its scales are then rewritten instead, and for
// few its codes into `codes` (else NULL); P is not read for r = 0.
struct Fp8Prep {
  int chunk, splits;
};
Fp8Prep fp8_prep_plan(int64_t M, int64_t C, bool few, int W = 1);
size_t fp8_rows_scale_bytes(int64_t M, int64_t C);
hipError_t launch_fp8_prep(const uint16_t* P, int64_t M, int64_t C, const uint16_t* Q, int r,
                           uint8_t* codes, uint8_t* scale, float* part, bool few, hipStream_t stream, bool f16, int W = 1,
                           const uint8_t* gcodes = nullptr, const uint8_t* gscale = nullptr);
// out = RN16([act | split] [f | fx]^T); f's scale byte of (output block,
// contraction block) at ob * fs_o + cb * fs_c. nn: f is [kc, nout up to 128].
// part: gemm_fp8_ws_bytes(). fp16 with kx > 0: row_scale as launch_scaled_columns'.
bool gemm_fp8_offsets_fit(int64_t M, int64_t kc, int kx, int64_t nout, bool nn);
size_t gemm_fp8_ws_bytes(int64_t M, int64_t kc, int64_t nout);
hipError_t launch_gemm_fp8(const uint8_t* act, const uint8_t* as, int64_t M, int64_t kc, const uint16_t* split, int kx,
                           const float* row_scale,
                           const uint8_t* f, const uint8_t* fs, int64_t fs_o, int64_t fs_c, int64_t fs_bytes,
                           const uint16_t* fx, int64_t nout, uint16_t* out, float* part, hipStream_t stream, bool f16,
                           bool nn);
// At most kGemvMostTokens tokens: Y = RN16(X8 W8^T + scale T B^T) from
// launch_fp8_prep's operands (few), or, up to 16 tokens, (rows) from codes [M, k up to
// 128] and scales [M, blocks] of each row; T as `parts` partials [parts][M][r] that the
// kernel adds in order, written to T_save if it is not NULL.
constexpr int64_t kGemvMostTokens = 64;
size_t fp8_gemv_codes_bytes(int64_t k, int64_t M);
size_t fp8_gemv_scale_bytes(int64_t k, int64_t M);
hipError_t launch_fp8_gemv(const Fp8View& w, const uint8_t* xq, const uint8_t* xs, bool rows, int64_t M, const float* T,
                           int parts, const uint16_t* B, int r, float scale, uint16_t* Y, float* T_save,
                           hipStream_t stream, bool f16);
// The values of activations encoded by row (qlora_fp8_rows), in 16 bits.
hipError_t launch_fp8_decode_rows(const uint8_t* codes, const uint8_t* scale, int64_t M, int64_t k, uint16_t* out,
                                  hipStream_t stream, bool f16);

// ---- residual addition and root-mean-square norm (rmsnorm.hip)
// R (with H) may be NULL, as may Y, rstd and codes (with scale; k % 64 == 0).
hipError_t launch_rms_fwd(const uint16_t* X, const uint16_t* R, const void* w, bool w32, int64_t M, int64_t k, float eps,
                          uint16_t* Y, uint16_t* H, float* rstd, uint8_t* codes, uint8_t* scale, hipStream_t stream,
                          bool f16);
// R, dX and dw may be NULL; part: rms_bwd_ws_bytes(M, k), for dw.
size_t rms_bwd_ws_bytes(int64_t M, int64_t k);
hipError_t launch_rms_bwd(const uint16_t* dY, const uint16_t* H, const float* rstd, const void* w, bool w32,
                          const uint16_t* R, int64_t M, int64_t k, uint16_t* dX, float* dw, int accumulate, float* part,
                          hipStream_t stream, bool f16);

hipError_t launch_silu_fwd(const uint16_t* G, const uint16_t* U, uint16_t* H, int64_t count,
                           hipStream_t stream);
hipError_t launch_silu_bwd(const uint16_t* G, const uint16_t* U, const uint16_t* dH, uint16_t* dG,
                           uint16_t* dU, int64_t count, hipStream_t stream);

}  // namespace qlora
