// The 8-bit layer's storage and operand layouts (internal; include/qlora.h
// states the public ones).
//
// Values are OCP E4M3 with a power-of-two scale 2^(b - 127) held as the
// exponent byte b, one per 128 consecutive contraction elements: of one row
// for activations, of 128 rows together for weights. b is the smallest byte
// whose scale brings the block's largest finite magnitude to at most 448, so
// nothing saturates, scaling is exact, and one rounding (to nearest, ties to
// even) is all that encoding does. gfx950's scaled MFMA multiplies by such
// scales inside the instruction: the product needs no vector work per block.
//
// What its sums hold (measured, scaled and unscaled forms alike): the products
// of 8 consecutive contraction elements are aligned at 2^-13 of the largest of
// them and cut off below, towards zero; the groups' sums add to the accumulator
// in fp32. That is 14 bits per group, an rms of 2^-16 of a sum of products of
// either sign, 2^-13.7 too little where all have one sign; the most it can be is
// 7 2^-13 of each group's largest product. The 8-bit rate comes with it; the
// rounding of an operand to 4 bits is about 2^10 times that rms, Y's to bf16 2^7.
#pragma once

#include "common.h"

namespace qlora {

constexpr int kF8Block = 128;

__host__ __device__ __forceinline__ int64_t f8_pad(int64_t c) { return (c + kF8Block - 1) / kF8Block * kF8Block; }

// Exponent byte for a block whose largest finite |x| has the fp32 bits
// `abits`: amax = 1.m 2^e needs 2^(e - 8) while 1.m <= 1.75 (448 = 1.75 2^8),
// else 2^(e - 7); bytes below 0 clamp (blocks under 2^-119), 0 takes scale 1.
__device__ __forceinline__ uint32_t f8_scale_byte(uint32_t abits) {
  const int e = (int)(abits >> 23) + ((abits & 0x7FFFFFu) > 0x600000u ? 1 : 0) - 8;
  return abits == 0 ? 127u : (uint32_t)(e < 0 ? 0 : e);
}

// 2^-(b - 127), exact for every byte f8_scale_byte gives (0 .. 247)
__device__ __forceinline__ float f8_inv_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// |x| as fp32 bits for the block maximum: 0 where x is not finite
__device__ __forceinline__ uint32_t f8_finite_abs(float x) {
  const uint32_t a = __float_as_uint(x) & 0x7FFFFFFFu;
  return a >= 0x7F800000u ? 0u : a;
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Largest of the 16 lanes of a row (lanes 16 q .. 16 q + 15), in all of them:
// rotations within the row by 8, 4, 2 and 1.
__device__ __forceinline__ uint32_t row16_max(uint32_t a) {
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x128, 0xF, 0xF, true));
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x124, 0xF, 0xF, true));
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x122, 0xF, 0xF, true));
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x121, 0xF, 0xF, true));
  return a;
}

// Four values times inv -> four E4M3 bytes. None is infinite: the callers
// have made NaN of infinities (the format has none), so that they stay visible
// in every product they enter.
__device__ __forceinline__ uint32_t f8_pack4(const float* x, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, w, true);
  return (uint32_t)w;
}

}  // namespace qlora
