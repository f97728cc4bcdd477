// Host side of the 8-bit layer's C ABI: argument checks, workspace carving
// and composition of its kernels.
#include <cmath>

#include "api_util.h"
#include "fp8.h"
#include "kernels.h"
#include "qlora.h"

using namespace qlora;

namespace {

qlora_status check_fp8(const qlora_fp8_weight* w) {
  if (w == nullptr) return QLORA_ERR_INVALID_ARG;
  if (w->n < 1 || w->k < 1 || w->k % QLORA_BLOCK != 0 || w->n > kMaxDim || w->k > kMaxDim) return QLORA_ERR_SHAPE;
  if (!good(w->codes) || !good(w->scale)) return QLORA_ERR_INVALID_ARG;
  return QLORA_OK;
}

Fp8View view8(const qlora_fp8_weight* w) { return Fp8View{w->n, w->k, w->codes, w->scale}; }

bool dims_ok(int64_t M, int64_t n, int64_t k, int r) {
  return M >= 0 && M <= kMaxDim && n >= 1 && n <= kMaxDim && k >= QLORA_BLOCK && k <= kMaxDim && k % QLORA_BLOCK == 0 &&
         r >= 0 && r <= QLORA_MAX_RANK;
}

// Whether the forward is one pass over the codes (else the GEMM); rows: the
// activations come encoded (qlora_fp8_rows), and two token tiles share a code.
// Four would need the pass twice: for weights up to 64 MB, which are in the
// last-level cache the second time. us, GEMM and pass, r = 64: 11008 x 4096 17 tokens
// 42 and 27, 64 tokens 44 and 37; 4096 x 4096 36 and 18, 39 and 21; 28672 x 8192 95 and 75,
// 99 and 113; 8192 x 28672 98 and 62, 104 and 98. The call that encodes takes the GEMM
// from 17 tokens on.
bool few_tokens(int64_t M, int64_t n, int64_t k, bool rows) {
  if (!rows || M <= 16) return M <= 16;
  return M <= 32 || (M <= kGemvMostTokens && n * f8_pad(k) <= (int64_t)64 << 20);
}

bool fwd_fits(int64_t M, int64_t n, int64_t k, int r, bool rows) {
  return few_tokens(M, n, k, rows) ? 32 * f8_pad(k) < ((int64_t)1 << 31)
                                   : gemm_fp8_offsets_fit(M, k, lora_extra_cols(r), n, false);
}

struct FwdWs {
  uint8_t* xq = nullptr;   // activation codes and scales
  uint8_t* xs = nullptr;
  float* proj = nullptr;   // partials of T
  float* T = nullptr;      // few tokens: T where its partials are too many for the GEMV to add
  uint16_t* TS = nullptr;  // low-rank operand columns
  float* rs = nullptr;     // their factor of each row (fp16)
  uint16_t* Bx = nullptr;
  uint16_t* Ao = nullptr;  // A in operand order
  float* part = nullptr;
};

// Few tokens: the GEMV adds T's partials itself while each of its workgroups
// reads at most 16 KB of them (1 - 2 us in the shadow of its first loads); a
// small kernel adds them before it otherwise (a launch, about 4 us).
bool gemv_adds(int64_t M, int64_t k, int r) { return (int64_t)fp8_prep_plan(M, k, true).splits * M * r * 4 <= 16384; }

// Few tokens that come encoded: whether the GEMV reads them by row. For r > 0
// the kernel before it brings them into operand order on its way (they cost the
// GEMV more by row: 11008 x 4096 at 16 tokens 14.9 us against 10), for r = 0
// that would be a launch of its own.
bool gemv_of_rows(int64_t M, int r) { return r == 0 && M <= 8; }

size_t fwd_ws(int64_t M, int64_t n, int64_t k, int r, bool rows, Carver& cv, FwdWs& o) {
  const bool few = few_tokens(M, n, k, rows);
  o.proj = cv.take<float>((size_t)fp8_prep_plan(M, k, few).splits * M * r * 4);
  if (few) {
    if (!rows || !gemv_of_rows(M, r)) o.xq = cv.take<uint8_t>(fp8_gemv_codes_bytes(k, M));
    if (!rows || !gemv_of_rows(M, r)) o.xs = cv.take<uint8_t>(fp8_gemv_scale_bytes(k, M));
    o.T = cv.take<float>((size_t)M * r * 4);
    return cv.used;
  }
  if (!rows) o.xq = cv.take<uint8_t>((size_t)M * f8_pad(k));
  o.xs = cv.take<uint8_t>(fp8_rows_scale_bytes(M, k));
  if (r > 0) {
    o.TS = cv.take<uint16_t>((size_t)M * lora_extra_cols(r) * 2);
    o.rs = cv.take<float>(row_scale_bytes(M));
    o.Bx = cv.take<uint16_t>((size_t)n * lora_extra_cols(r) * 2);
    o.Ao = cv.take<uint16_t>(operand_order_bytes(f8_pad(k), r));
  }
  o.part = cv.take<float>(gemm_fp8_ws_bytes(M, k, n));
  return cv.used;
}

struct BwdWs {
  uint8_t* yq = nullptr;   // dY's codes and scale words
  uint8_t* ys = nullptr;
  uint16_t* US = nullptr;
  float* rs = nullptr;     // the factor of each row of US (fp16)
  uint16_t* Ax = nullptr;
  uint16_t* Bo = nullptr;  // B in operand order
  float* U = nullptr;
  float* T = nullptr;
  float* proj = nullptr;
  void* Up = nullptr;      // U's and T's parts
  void* Tp = nullptr;
  float* da = nullptr;     // partials of the gradients
  float* db = nullptr;
  float* part = nullptr;
};

size_t bwd_ws(int64_t M, int64_t n, int64_t k, int r, Carver& cv, BwdWs& o) {
  o.yq = cv.take<uint8_t>((size_t)M * f8_pad(n));
  o.ys = cv.take<uint8_t>(fp8_rows_scale_bytes(M, n));
  if (r > 0) {
    o.US = cv.take<uint16_t>((size_t)M * lora_extra_cols(r) * 2);
    o.rs = cv.take<float>(row_scale_bytes(M));
    o.Ax = cv.take<uint16_t>((size_t)k * lora_extra_cols(r) * 2);
    o.Bo = cv.take<uint16_t>(operand_order_bytes(f8_pad(n), r));
    o.U = cv.take<float>((size_t)M * r * 4);
    o.T = cv.take<float>((size_t)M * r * 4);
    const size_t p1 = (size_t)fp8_prep_plan(M, n, false).splits * M * r * 4, p2 = rowdot_ws_bytes(M, k, r);
    o.proj = cv.take<float>(p1 > p2 ? p1 : p2);
    o.Up = cv.take<char>(rank_parts_bytes(M, r, 1));
    o.Tp = cv.take<char>(rank_parts_bytes(M, r, 1));
    o.da = cv.take<float>(colgrad_ws_bytes(M, k, r, 1));
    o.db = cv.take<float>(colgrad_ws_bytes(M, n, r, 1));
  }
  o.part = cv.take<float>(gemm_fp8_ws_bytes(M, n, k));
  return cv.used;
}

bool is16(int dtype) { return dtype == QLORA_DT_BF16 || dtype == QLORA_DT_FP16; }

// The forward; x8: the activations' codes and scales, or NULL where X is encoded here.
qlora_status fwd_impl(const qlora_fp8_weight* w, const qlora_fp8_rows* x8, const void* X, int64_t M, int dtype,
                      const void* A, const void* B, int r, float scale, void* Y, float* T_save, void* ws, size_t ws_bytes,
                      void* stream) {
  const bool rows = x8 != nullptr;
  const int64_t n = w->n, k = w->k;
  if (!is16(dtype)) return QLORA_ERR_INVALID_ARG;
  if (!dims_ok(M, n, k, r) || !fwd_fits(M, n, k, r, rows)) return QLORA_ERR_SHAPE;
  if (M == 0) return QLORA_OK;
  if (((!rows || r > 0) && !good(X)) || !good(Y) || (r > 0 && (!good(A) || !good(B))) || (T_save && !aligned16(T_save)))
    return QLORA_ERR_INVALID_ARG;
  if (rows && (!good(x8->codes) || !good(x8->scale))) return QLORA_ERR_INVALID_ARG;
  Carver size(nullptr), cv(ws);
  FwdWs o;
  const size_t need = fwd_ws(M, n, k, r, rows, size, o);
  if (need > 0 && (!good(ws) || ws_bytes < need)) return QLORA_ERR_WORKSPACE;
  fwd_ws(M, n, k, r, rows, cv, o);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool f16 = dtype == QLORA_DT_FP16;
  const uint16_t *x = static_cast<const uint16_t*>(X), *a = static_cast<const uint16_t*>(A),
                 *b = static_cast<const uint16_t*>(B);
  const bool few = few_tokens(M, n, k, rows);
  const int parts = fp8_prep_plan(M, k, few).splits;
  hipError_t e = hipSuccess;
  if (r > 0 && !few) e = launch_factors(a, 0, k, f8_pad(k), r, o.Ao, b, n, o.Bx, st);
  const bool by_row = rows && few && gemv_of_rows(M, r);
  if (e == hipSuccess && !by_row)
    e = launch_fp8_prep(x, M, k, few ? a : o.Ao, r, o.xq, o.xs, o.proj, few, st, f16, 1, rows ? x8->codes : nullptr,
                        rows ? x8->scale : nullptr);
  const uint8_t* const xq = by_row || (rows && !few) ? x8->codes : o.xq;
  const uint8_t* const xs = by_row ? x8->scale : o.xs;
  if (few) {
    if (r > 0 && !gemv_adds(M, k, r)) {
      float* const T = T_save ? T_save : o.T;
      if (e == hipSuccess) e = launch_rowdot_finalize(o.proj, parts, M, r, T, nullptr, scale, st, f16);
      if (e == hipSuccess)
        e = launch_fp8_gemv(view8(w), xq, xs, by_row, M, T, 1, b, r, scale, static_cast<uint16_t*>(Y), nullptr, st, f16);
    } else if (e == hipSuccess) {
      e = launch_fp8_gemv(view8(w), xq, xs, by_row, M, o.proj, parts, b, r, scale, static_cast<uint16_t*>(Y), T_save, st, f16);
    }
    return hip_status(e);
  }
  const int64_t nb = f8_pad(k) / kF8Block;
  if (r > 0 && e == hipSuccess)
    e = f16 ? launch_scaled_columns(o.proj, parts, 1, M, r, lora_extra_cols(r), scale, T_save, o.TS, o.rs, st)
            : launch_rowdot_finalize(o.proj, parts, M, r, T_save, o.TS, scale, st, false);
  if (e == hipSuccess)
    e = launch_gemm_fp8(xq, o.xs, M, k, o.TS, lora_extra_cols(r), o.rs, w->codes, w->scale, nb, 1,
                        (f8_pad(n) / kF8Block) * nb, o.Bx, n, static_cast<uint16_t*>(Y), o.part, st, f16, false);
  return hip_status(e);
}

}  // namespace

extern "C" {

size_t qlora_fp8_storage_bytes(int64_t n, int64_t k) {
  if (n < 1 || k < 1 || k % QLORA_BLOCK) return 0;
  return (size_t)(n * f8_pad(k) + (f8_pad(n) / kF8Block) * (f8_pad(k) / kF8Block));
}

qlora_status qlora_quantize_fp8(const void* W, int w_dtype, const qlora_fp8_weight* out, void* stream) {
  const qlora_status s = check_fp8(out);
  if (s != QLORA_OK) return s;
  if (w_dtype != QLORA_DT_FP32 && !is16(w_dtype)) return QLORA_ERR_INVALID_ARG;
  if (!good(W)) return QLORA_ERR_INVALID_ARG;
  return hip_status(
      launch_fp8_encode(W, w_dtype, out->n, out->k, out->codes, out->scale, static_cast<hipStream_t>(stream)));
}

qlora_status qlora_dequant_fp8(const qlora_fp8_weight* w, void* out, void* stream) {
  const qlora_status s = check_fp8(w);
  if (s != QLORA_OK) return s;
  if (!good(out)) return QLORA_ERR_INVALID_ARG;
  return hip_status(launch_fp8_decode(view8(w), static_cast<uint16_t*>(out), static_cast<hipStream_t>(stream)));
}

size_t qlora_fp8_linear_workspace_bytes(int64_t M, int64_t n, int64_t k, int r, int is_bwd) {
  if (M < 1 || !dims_ok(M, n, k, r) || (is_bwd != 0 && is_bwd != 1)) return 0;
  Carver cv(nullptr);
  if (is_bwd) {
    BwdWs o;
    return bwd_ws(M, n, k, r, cv, o);
  }
  FwdWs o;
  return fwd_ws(M, n, k, r, false, cv, o);
}

qlora_status qlora_fp8_linear_fwd(const qlora_fp8_weight* w, const void* X, int64_t M, int dtype, const void* A,
                                  const void* B, int r, float scale, void* Y, float* T_save, void* ws, size_t ws_bytes,
                                  void* stream) {
  const qlora_status s = check_fp8(w);
  if (s != QLORA_OK) return s;
  return fwd_impl(w, nullptr, X, M, dtype, A, B, r, scale, Y, T_save, ws, ws_bytes, stream);
}

size_t qlora_fp8_rows_bytes(int64_t M, int64_t k) {
  if (M < 1 || k < 1 || k % QLORA_BLOCK) return 0;
  return (size_t)(M * f8_pad(k) + M * (f8_pad(k) / kF8Block));
}

qlora_status qlora_dequant_fp8_rows(const qlora_fp8_rows* x, int dtype, void* out, void* stream) {
  if (x == nullptr || !is16(dtype)) return QLORA_ERR_INVALID_ARG;
  if (x->M < 0 || x->M > kMaxDim || x->k < 1 || x->k > kMaxDim || x->k % QLORA_BLOCK) return QLORA_ERR_SHAPE;
  if (x->M == 0) return QLORA_OK;
  if (!good(x->codes) || !good(x->scale) || !good(out)) return QLORA_ERR_INVALID_ARG;
  return hip_status(launch_fp8_decode_rows(x->codes, x->scale, x->M, x->k, static_cast<uint16_t*>(out),
                                           static_cast<hipStream_t>(stream), dtype == QLORA_DT_FP16));
}

size_t qlora_fp8_linear_rows_workspace_bytes(int64_t M, int64_t n, int64_t k, int r) {
  if (M < 1 || !dims_ok(M, n, k, r)) return 0;
  Carver cv(nullptr);
  FwdWs o;
  return fwd_ws(M, n, k, r, true, cv, o);
}

qlora_status qlora_fp8_linear_fwd_rows(const qlora_fp8_weight* w, const qlora_fp8_rows* x8, const void* X, int dtype,
                                       const void* A, const void* B, int r, float scale, void* Y, float* T_save,
                                       void* ws, size_t ws_bytes, void* stream) {
  const qlora_status s = check_fp8(w);
  if (s != QLORA_OK) return s;
  if (x8 == nullptr) return QLORA_ERR_INVALID_ARG;
  if (x8->k != w->k) return QLORA_ERR_SHAPE;
  return fwd_impl(w, x8, X, x8->M, dtype, A, B, r, scale, Y, T_save, ws, ws_bytes, stream);
}

qlora_status qlora_fp8_linear_bwd(const qlora_fp8_weight* w, const void* X, const float* T_saved, const void* dY,
                                  int64_t M, int dtype, const void* A, const void* B, int r, float scale, void* dX,
                                  float* dA, float* dB, int accumulate, void* ws, size_t ws_bytes, void* stream) {
  const qlora_status s = check_fp8(w);
  if (s != QLORA_OK) return s;
  const int64_t n = w->n, k = w->k;
  if (!is16(dtype) || (accumulate != 0 && accumulate != 1)) return QLORA_ERR_INVALID_ARG;
  if (!dims_ok(M, n, k, r) || (M > 0 && dX && !gemm_fp8_offsets_fit(M, n, lora_extra_cols(r), k, true)))
    return QLORA_ERR_SHAPE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (r == 0) {
    dA = nullptr;
    dB = nullptr;
  }
  if ((dX && !aligned16(dX)) || (dA && !aligned16(dA)) || (dB && !aligned16(dB))) return QLORA_ERR_INVALID_ARG;
  hipError_t e = hipSuccess;
  if (M == 0) {
    if (accumulate) return QLORA_OK;
    if (dA) e = zero_f32(dA, (int64_t)r * k, st);
    if (e == hipSuccess && dB) e = zero_f32(dB, n * (int64_t)r, st);
    return hip_status(e);
  }
  const bool need_x = dA != nullptr || (dB != nullptr && T_saved == nullptr);
  if (!good(dY) || (need_x && !good(X)) || (r > 0 && (!good(A) || !good(B))) || (T_saved && !aligned16(T_saved)))
    return QLORA_ERR_INVALID_ARG;
  if (!good(ws) || ws_bytes < qlora_fp8_linear_workspace_bytes(M, n, k, r, 1)) return QLORA_ERR_WORKSPACE;
  Carver cv(ws);
  BwdWs o;
  bwd_ws(M, n, k, r, cv, o);
  const bool f16 = dtype == QLORA_DT_FP16;
  const uint16_t *x = static_cast<const uint16_t*>(X), *dy = static_cast<const uint16_t*>(dY),
                 *a = static_cast<const uint16_t*>(A), *b = static_cast<const uint16_t*>(B);
  if (dX || dA) {
    if (r > 0 && dX)
      e = launch_factors(b, 1, n, f8_pad(n), r, o.Bo, a, k, o.Ax, st);
    else if (r > 0)
      e = launch_operand_order(b, nullptr, 1, n, f8_pad(n), r, o.Bo, st);
    if (e == hipSuccess)
      e = launch_fp8_prep(dy, M, n, o.Bo, r, dX ? o.yq : nullptr, o.ys, o.proj, false, st, f16);
    const int parts = fp8_prep_plan(M, n, false).splits;
    uint16_t* const us = dX ? o.US : nullptr;
    if (e == hipSuccess && r > 0)
      e = f16 ? launch_scaled_columns(o.proj, parts, 1, M, r, lora_extra_cols(r), scale, o.U, us, o.rs, st)
              : launch_rowdot_finalize(o.proj, parts, M, r, o.U, us, scale, st, false);
  }
  if (dX) {
    const int64_t kb = f8_pad(k) / kF8Block;
    if (e == hipSuccess)
      e = launch_gemm_fp8(o.yq, o.ys, M, n, o.US, lora_extra_cols(r), o.rs, w->codes, w->scale, 1, kb,
                          (f8_pad(n) / kF8Block) * kb, o.Ax, k, static_cast<uint16_t*>(dX), o.part, st, f16, true);
  }
  if (!dA && !dB) return hip_status(e);
  const float* T = T_saved;
  if (e == hipSuccess && dB && T == nullptr) {
    e = launch_rowdot(x, M, k, a, 0, r, o.T, nullptr, scale, o.proj, st, nullptr, f16);
    T = o.T;
  }
  GradJob ja{}, jb{};
  if (e == hipSuccess) e = launch_rank_parts(o.U, dA ? 1 : 0, o.Up, T, dB ? 1 : 0, o.Tp, M, r, st);
  if (e == hipSuccess && dA)
    e = launch_colgrad(x, M, k, o.Up, 1, r, scale, dA, nullptr, true, accumulate, o.da, ja, st, f16);
  if (e == hipSuccess && dB)
    e = launch_colgrad(dy, M, n, o.Tp, 1, r, scale, dB, nullptr, false, accumulate, o.db, jb, st, f16);
  if (e == hipSuccess) e = launch_grad_reduce(ja, jb, scale, accumulate, st);
  return hip_status(e);
}

}  // extern "C"
