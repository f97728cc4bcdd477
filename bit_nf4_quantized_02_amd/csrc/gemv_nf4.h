// Pieces of the small-token-count kernels over NF4 weights (gemv_nf4.hip,
// gemv_pair.hip).
#pragma once

#include "common.h"

#ifndef QLORA_GEMV_XP_MIN_M
#define QLORA_GEMV_XP_MIN_M 5
#endif

namespace qlora {

// s_waitcnt immediate that waits for LDS / scalar-memory operations only
// (lgkmcnt <= n; vmcnt and expcnt left at their maxima)
constexpr int lgkm_wait(int n) { return 0xC07F | (n << 8); }

// Swizzle of a 128-byte code line in LDS: row r of a 16-row tile keeps its
// 16-byte segment g at position g ^ sw(r). The 8 (or 16) lanes that read one
// segment of 8 (16) consecutive rows in one LDS cycle then hit distinct banks
// whether the LDS serves 128 or 256 bytes per cycle.
__device__ __forceinline__ int code_swz(int r) { return (r ^ (r >> 3)) & 7; }

// Scale fields of block blk in one of the three stored forms, without
// branches (kForm 0: double-quantized, E4M3 code + fp32 second-level scale
// per 256 blocks; 1: fp32 per block; 2: bf16 per block), as scale_fields.
// c8r / s2r: descriptors of the code and scale arrays.
template <int kForm>
__device__ __forceinline__ void scale_fields_of(const i32x4& c8r, const i32x4& s2r, uint32_t blk, uint32_t& c8,
                                                float& s2v) {
  if constexpr (kForm == 0) {
    c8 = raw_buffer_load_u8(c8r, (int)blk, 0, 0);
    s2v = __builtin_bit_cast(float, raw_buffer_load_u32(s2r, (int)((blk / kDqBlock) * 4), 0, 0));
  } else if constexpr (kForm == 1) {
    c8 = kE4m3One;
    s2v = __builtin_bit_cast(float, raw_buffer_load_u32(s2r, (int)(blk * 4), 0, 0));
  } else {
    c8 = kE4m3One;
    s2v = bf16_bits_to_f32(raw_buffer_load_u16(s2r, (int)(blk * 2), 0, 0));
  }
}

// Token counts from which the activations are first rewritten in operand
// order: below it the few distinct rows an activation load touches cost less
// than the extra pass (measured on the 70B-class shapes). Weights with fewer
// than kXpMinN rows never take it: their workgroups re-read X only a few
// times, and the extra launch costs more (a 1024 x 1024 layer at M = 16).
constexpr int64_t kXpMinM = QLORA_GEMV_XP_MIN_M;
constexpr int64_t kXpMinN = 4096;
inline bool gemv_orders_x(int64_t M, int64_t n) { return M >= kXpMinM && n >= kXpMinN; }

}  // namespace qlora
