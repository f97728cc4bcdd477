// Host side of the gated feed-forward block's C ABI: argument checks,
// workspace carving and composition of its kernels.
#include "api_util.h"
#include "kernels.h"
#include "qlora.h"

using namespace qlora;

namespace {

// Both weights valid, of one shape and one storage form.
qlora_status check_pair(const qlora_nf4_weight* g, const qlora_nf4_weight* u) {
  qlora_status s = check_weight(g);
  if (s == QLORA_OK) s = check_weight(u);
  if (s != QLORA_OK) return s;
  if (g->n != u->n || g->k != u->k || g->n > kMaxDim || g->k > kMaxDim) return QLORA_ERR_SHAPE;
  if ((g->code8 == nullptr) != (u->code8 == nullptr) || g->scale_bf16 != u->scale_bf16) return QLORA_ERR_INVALID_ARG;
  return QLORA_OK;
}

bool dims_ok(int64_t M, int64_t n, int64_t k, int r) {
  return M >= 0 && M <= kMaxDim && n >= 1 && n <= kMaxDim && k >= QLORA_BLOCK && k <= kMaxDim && k % QLORA_BLOCK == 0 &&
         r >= 0 && r <= QLORA_MAX_RANK;
}

bool is16(int dtype) { return dtype == QLORA_DT_BF16 || dtype == QLORA_DT_FP16; }

bool few_tokens(int64_t M, int64_t n, int64_t k) { return M <= 16 && gemv_fits(n, k); }

bool fwd_fits(int64_t M, int64_t n, int64_t k, int r) {
  return few_tokens(M, n, k) || gemm_bf16_offsets_fit(M, k, gated_extra_cols(r), gated_rows(n));
}

bool dx_fits(int64_t M, int64_t n, int64_t k, int r) {
  const int64_t kc = 2 * gated_pad(n);
  const int xc = gated_extra_cols(r);
  return gemm_bf16_offsets_fit(M, kc, xc, k) && (kc + xc) * k * 2 < ((int64_t)1 << 32);
}

struct FwdWs {
  void* few = nullptr;     // few tokens: the GEMV's operands
  void* proj = nullptr;
  uint16_t* TS = nullptr;  // low-rank columns of the GEMM
  float* rs = nullptr;     // their factor of each row (fp16)
  uint16_t* F = nullptr;   // both weights expanded
  float* part = nullptr;
};

size_t fwd_ws(int64_t M, int64_t n, int64_t k, int r, Carver& cv, FwdWs& o) {
  if (few_tokens(M, n, k)) {
    o.few = cv.take<char>(gemv_pair_ws_bytes(M, n, k, r));
    return cv.used;
  }
  const int xc = gated_extra_cols(r);
  if (r > 0) o.proj = cv.take<char>(gated_project_ws_bytes(M, k, r));
  if (r > 0) o.TS = cv.take<uint16_t>((size_t)M * xc * 2);
  if (r > 0) o.rs = cv.take<float>(row_scale_bytes(M, 2));
  o.F = cv.take<uint16_t>(gated_fwd_operand_bytes(n, k, r));
  o.part = cv.take<float>(gemm_bf16_ws_bytes(M, k, xc, gated_rows(n)));
  return cv.used;
}

struct BwdWs {
  float* T = nullptr;      // [2][M][r] without T_saved
  float* P = nullptr;      // [2][M][r]
  uint16_t* PS = nullptr;  // low-rank columns of dX's GEMM
  float* rs = nullptr;     // their factor of each row (fp16)
  uint16_t* D = nullptr;   // [dG | dU]
  uint16_t* F = nullptr;   // both weights, contraction-major
  void* proj = nullptr;
  void* join = nullptr;
  void* Pp = nullptr;      // P's and T's parts
  void* Tp = nullptr;
  float* da = nullptr;     // partials of the gradients
  float* db = nullptr;
  float* part = nullptr;
};

size_t bwd_ws(int64_t M, int64_t n, int64_t k, int r, Carver& cv, BwdWs& o) {
  const int xc = gated_extra_cols(r);
  const int64_t np = gated_pad(n);
  if (r > 0) {
    o.T = cv.take<float>((size_t)2 * M * r * 4);
    o.P = cv.take<float>((size_t)2 * M * r * 4);
    o.PS = cv.take<uint16_t>((size_t)M * xc * 2);
    o.rs = cv.take<float>(row_scale_bytes(M));
    o.proj = cv.take<char>(gated_project_ws_bytes(M, k, r));
    o.join = cv.take<char>(gated_join_ws_bytes(M, n, r));
    o.Pp = cv.take<char>(rank_parts_bytes(M, r, 2));
    o.Tp = cv.take<char>(rank_parts_bytes(M, r, 2));
    o.da = cv.take<float>(colgrad_ws_bytes(M, k, r, 2));
    o.db = cv.take<float>(gated_db_ws_bytes(M, n, r));
  }
  o.D = cv.take<uint16_t>((size_t)M * 2 * np * 2);
  o.F = cv.take<uint16_t>(gated_dx_operand_bytes(n, k, r));
  o.part = cv.take<float>(gemm_bf16_ws_bytes(M, 2 * np, xc, k));
  return cv.used;
}

const uint16_t* u16(const void* p) { return static_cast<const uint16_t*>(p); }

}  // namespace

extern "C" {

size_t qlora_gated_workspace_bytes(int64_t M, int64_t n, int64_t k, int r, int is_bwd) {
  if (M < 1 || !dims_ok(M, n, k, r) || (is_bwd != 0 && is_bwd != 1)) return 0;
  Carver cv(nullptr);
  if (is_bwd) {
    BwdWs o;
    return bwd_ws(M, n, k, r, cv, o);
  }
  FwdWs o;
  return fwd_ws(M, n, k, r, cv, o);
}

qlora_status qlora_gated_fwd(const qlora_nf4_weight* w_gate, const qlora_nf4_weight* w_up, const void* X, int64_t M,
                             int dtype, const void* A_gate, const void* B_gate, const void* A_up, const void* B_up,
                             int r, float scale, void* H, void* G_save, void* U_save, float* T_save, void* ws,
                             size_t ws_bytes, void* stream) {
  const qlora_status s = check_pair(w_gate, w_up);
  if (s != QLORA_OK) return s;
  const int64_t n = w_gate->n, k = w_gate->k;
  if (!is16(dtype)) return QLORA_ERR_INVALID_ARG;
  if (!dims_ok(M, n, k, r) || !fwd_fits(M, n, k, r)) return QLORA_ERR_SHAPE;
  if (M == 0) return QLORA_OK;
  if (!good(X) || !good(H) || (G_save && !aligned16(G_save)) || (U_save && !aligned16(U_save)) ||
      (T_save && !aligned16(T_save)))
    return QLORA_ERR_INVALID_ARG;
  if (r > 0 && (!good(A_gate) || !good(B_gate) || !good(A_up) || !good(B_up))) return QLORA_ERR_INVALID_ARG;
  if (!good(ws) || ws_bytes < qlora_gated_workspace_bytes(M, n, k, r, 0)) return QLORA_ERR_WORKSPACE;
  Carver cv(ws);
  FwdWs o;
  fwd_ws(M, n, k, r, cv, o);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool f16 = dtype == QLORA_DT_FP16;
  const Nf4View g = view_of(w_gate), u = view_of(w_up);
  const uint16_t* const x = u16(X);
  uint16_t *const h = static_cast<uint16_t*>(H), *const gs = static_cast<uint16_t*>(G_save),
           *const us = static_cast<uint16_t*>(U_save);
  if (few_tokens(M, n, k))
    return hip_status(launch_gemv_pair(g, u, x, M, u16(A_gate), u16(B_gate), u16(A_up), u16(B_up), r, scale, h, gs, us,
                                       T_save, o.few, st, f16));
  hipError_t e = hipSuccess;
  const int xc = gated_extra_cols(r);
  if (r > 0) e = launch_gated_project(x, M, k, u16(A_gate), u16(A_up), r, scale, T_save, o.TS, o.rs, o.proj,
                                    st, f16);
  if (e == hipSuccess) e = launch_gated_expand_fwd(g, u, u16(B_gate), u16(B_up), r, o.F, st, f16);
  if (e == hipSuccess) e = launch_gemm_gated(x, M, k, o.TS, xc, o.rs, o.F, n, h, gs, us, o.part, st, f16);
  return hip_status(e);
}

qlora_status qlora_gated_bwd(const qlora_nf4_weight* w_gate, const qlora_nf4_weight* w_up, const void* X,
                             const float* T_saved, const void* G, const void* U, const void* dH, int64_t M, int dtype,
                             const void* A_gate, const void* B_gate, const void* A_up, const void* B_up, int r,
                             float scale, void* dX, float* dA_gate, float* dB_gate, float* dA_up, float* dB_up,
                             int accumulate, void* ws, size_t ws_bytes, void* stream) {
  const qlora_status s = check_pair(w_gate, w_up);
  if (s != QLORA_OK) return s;
  const int64_t n = w_gate->n, k = w_gate->k;
  if (!is16(dtype) || (accumulate != 0 && accumulate != 1)) return QLORA_ERR_INVALID_ARG;
  if (!dims_ok(M, n, k, r) || (dX && !dx_fits(M, n, k, r))) return QLORA_ERR_SHAPE;
  if (r == 0) dA_gate = dB_gate = dA_up = dB_up = nullptr;
  if ((dX && !aligned16(dX)) || (dA_gate && !aligned16(dA_gate)) || (dB_gate && !aligned16(dB_gate)) ||
      (dA_up && !aligned16(dA_up)) || (dB_up && !aligned16(dB_up)))
    return QLORA_ERR_INVALID_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (M == 0) {
    if (accumulate) return QLORA_OK;
    for (float* p : {dA_gate, dA_up})
      if (e == hipSuccess && p) e = zero_f32(p, (int64_t)r * k, st);
    for (float* p : {dB_gate, dB_up})
      if (e == hipSuccess && p) e = zero_f32(p, n * (int64_t)r, st);
    return hip_status(e);
  }
  const bool need_a = dA_gate || dA_up, need_b = dB_gate || dB_up;
  if (!good(G) || !good(U) || !good(dH) || (T_saved && !aligned16(T_saved))) return QLORA_ERR_INVALID_ARG;
  if ((need_a || (need_b && !T_saved)) && !good(X)) return QLORA_ERR_INVALID_ARG;
  if (r > 0 && (!good(A_gate) || !good(B_gate) || !good(A_up) || !good(B_up))) return QLORA_ERR_INVALID_ARG;
  if (!good(ws) || ws_bytes < qlora_gated_workspace_bytes(M, n, k, r, 1)) return QLORA_ERR_WORKSPACE;
  Carver cv(ws);
  BwdWs o;
  bwd_ws(M, n, k, r, cv, o);
  const bool f16 = dtype == QLORA_DT_FP16;
  const int xc = gated_extra_cols(r);
  const int64_t np = gated_pad(n);
  const uint16_t* const x = u16(X);
  if (dX || need_a)
    e = launch_gated_join(u16(G), u16(U), u16(dH), M, n, u16(B_gate), u16(B_up), r, scale, dX ? o.D : nullptr, o.P,
                          dX ? o.PS : nullptr, o.rs, o.join, st, f16);
  if (dX) {
    if (e == hipSuccess)
      e = launch_gated_expand_dx(view_of(w_gate), view_of(w_up), u16(A_gate), u16(A_up), r, o.F, st, f16);
    if (e == hipSuccess)
      e = launch_gemm_bf16_ext(o.D, M, 2 * np, r > 0 ? o.PS : nullptr, xc, o.F, k, o.F + 2 * np * k, k, k,
                               static_cast<uint16_t*>(dX), o.part, st, nullptr, 1.0f, f16, /*nn=*/true,
                               o.rs);
  }
  if (!need_a && !need_b) return hip_status(e);
  const float* T = T_saved;
  if (e == hipSuccess && need_b && T == nullptr) {
    e = launch_gated_project(x, M, k, u16(A_gate), u16(A_up), r, scale, o.T, nullptr, nullptr, o.proj, st,
                             f16);
    T = o.T;
  }
  GradJob ja{}, jb{};
  if (e == hipSuccess) e = launch_rank_parts(o.P, need_a ? 2 : 0, o.Pp, T, need_b ? 2 : 0, o.Tp, M, r, st);
  if (e == hipSuccess && need_a)
    e = launch_colgrad(x, M, k, o.Pp, 2, r, scale, dA_gate, dA_up, true, accumulate, o.da, ja, st, f16);
  if (e == hipSuccess && need_b)
    e = launch_gated_db(u16(G), u16(U), u16(dH), M, n, o.Tp, r, dB_gate, dB_up, o.db, jb, st, f16);
  if (e == hipSuccess) e = launch_grad_reduce(ja, jb, scale, accumulate, st);
  return hip_status(e);
}

}  // extern "C"
