// Host side of the norm's C ABI: argument checks and launches.
#include <cmath>

#include "api_util.h"
#include "fp8.h"
#include "kernels.h"
#include "qlora.h"

using namespace qlora;

namespace {

bool is16(int dtype) { return dtype == QLORA_DT_BF16 || dtype == QLORA_DT_FP16; }

// The gain's type: the activations' or fp32.
bool gain_ok(int w_dtype, int dtype) { return w_dtype == dtype || w_dtype == QLORA_DT_FP32; }

bool dims_ok(int64_t M, int64_t k) {
  return M >= 0 && M <= kMaxDim && k >= 1 && k <= kMaxDim && M * k <= ((int64_t)1 << 36);
}

bool eps_ok(float eps) { return eps >= 0.0f && !std::isinf(eps); }

}  // namespace

extern "C" {

qlora_status qlora_rms_norm_fwd(const void* X, const void* residual, const void* w, int w_dtype, int64_t M, int64_t k,
                                int dtype, float eps, void* Y, void* H, float* rstd, const qlora_fp8_rows* X8,
                                void* stream) {
  if (!is16(dtype) || !gain_ok(w_dtype, dtype) || !eps_ok(eps)) return QLORA_ERR_INVALID_ARG;
  if (!dims_ok(M, k)) return QLORA_ERR_SHAPE;
  if (X8 != nullptr && (X8->M != M || X8->k != k || k % QLORA_BLOCK != 0)) return QLORA_ERR_SHAPE;
  if (M == 0) return QLORA_OK;
  if (!good(X) || !good(w) || !aligned16(residual) || !aligned16(Y) || !aligned16(rstd)) return QLORA_ERR_INVALID_ARG;
  if ((residual != nullptr) != (H != nullptr) || !aligned16(H)) return QLORA_ERR_INVALID_ARG;
  if (X8 != nullptr && (!good(X8->codes) || !good(X8->scale))) return QLORA_ERR_INVALID_ARG;
  return hip_status(launch_rms_fwd(static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(residual), w,
                                   w_dtype == QLORA_DT_FP32, M, k, eps, static_cast<uint16_t*>(Y),
                                   static_cast<uint16_t*>(H), rstd, X8 ? X8->codes : nullptr, X8 ? X8->scale : nullptr,
                                   static_cast<hipStream_t>(stream), dtype == QLORA_DT_FP16));
}

size_t qlora_rms_norm_bwd_workspace_bytes(int64_t M, int64_t k) {
  return M >= 1 && dims_ok(M, k) ? rms_bwd_ws_bytes(M, k) : 0;
}

qlora_status qlora_rms_norm_bwd(const void* dY, const void* H, const float* rstd, const void* w, int w_dtype,
                                const void* dres, int64_t M, int64_t k, int dtype, void* dX, float* dw, int accumulate,
                                void* ws, size_t ws_bytes, void* stream) {
  if (!is16(dtype) || !gain_ok(w_dtype, dtype) || (accumulate != 0 && accumulate != 1)) return QLORA_ERR_INVALID_ARG;
  if (!dims_ok(M, k)) return QLORA_ERR_SHAPE;
  if (!aligned16(dX) || !aligned16(dw)) return QLORA_ERR_INVALID_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (M == 0) return dw && !accumulate ? hip_status(zero_f32(dw, k, st)) : QLORA_OK;
  if (!good(dY) || !good(H) || !good(rstd) || !good(w) || !aligned16(dres)) return QLORA_ERR_INVALID_ARG;
  if (dX == nullptr && dw == nullptr) return QLORA_OK;
  if (dw != nullptr && (!good(ws) || ws_bytes < qlora_rms_norm_bwd_workspace_bytes(M, k))) return QLORA_ERR_WORKSPACE;
  return hip_status(launch_rms_bwd(static_cast<const uint16_t*>(dY), static_cast<const uint16_t*>(H), rstd, w,
                                   w_dtype == QLORA_DT_FP32, static_cast<const uint16_t*>(dres), M, k,
                                   static_cast<uint16_t*>(dX), dw, accumulate, static_cast<float*>(ws), st,
                                   dtype == QLORA_DT_FP16));
}

}  // extern "C"
