// Pieces of the gradient kernels (gated.hip's join and dB, colgrad.hip): fp32
// values in 16-bit parts, and the staged tile whose columns come back as MFMA
// operands.
#pragma once

#include "common.h"

namespace qlora {

// Eight fp32 values -> kN bf16 parts whose sum holds 8 kN bits of each. bf16
// for both compute types: its exponents are fp32's, so three parts hold all 24
// bits of a gradient of any size, where the second of two fp16 parts is below
// fp16's smallest step for values under 2^-3 (2e-3 of the sum lost at 1e-5) and
// the first infinite above 65504. Two parts hold an fp16 value exactly (11 bits).
constexpr int kParts = 3;

template <int kN>
__device__ __forceinline__ void split8(const float (&x)[8], u32x4 (&p)[kN]) {
  float rem[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    rem[e] = x[e];
    // one fp32 value from here on: folded into the operation that made x, the
    // conversion stored and the one subtracted could be rounded from different values
    asm("" : "+v"(rem[e]));
  }
#pragma unroll
  for (int q = 0; q < kN; ++q)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      p[q][w] = pack2<false>(rem[2 * w], rem[2 * w + 1]);
      asm("" : "+v"(p[q][w]));  // (unpacked from here, not converted a second time)
      rem[2 * w] -= from16<false>(p[q][w] & 0xFFFFu);
      rem[2 * w + 1] -= from16<false>(p[q][w] >> 16);
    }
}

// Eight 16-bit values -> bf16 parts: themselves, or an fp16 value's two.
template <bool kF16>
constexpr int parts16() { return kF16 ? 2 : 1; }

template <bool kF16>
__device__ __forceinline__ void split8h(const u32x4& v, u32x4 (&p)[parts16<kF16>()]) {
  if constexpr (kF16) {
    float x[8];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      x[2 * w] = from16<true>(v[w] & 0xFFFFu);
      x[2 * w + 1] = from16<true>(v[w] >> 16);
    }
    split8(x, p);
  } else {
    p[0] = v;
  }
}

// Columns of a workgroup, and bytes of a staged tile [32 tokens][64 columns].
constexpr int kDbCols = 64;
constexpr int kDbTile = 32 * kDbCols * 2;

// In a staged tile the 32-byte segment s of row i is kept
// at s ^ f(i), f(i) = bit 1 of i + 2 (bit 3 of i), so that the eight rows that
// one cycle of a transposing read touches lie on distinct banks.
__device__ __forceinline__ int db_seg(int row, int s) { return row * 128 + ((s ^ (((row >> 1) & 1) | ((row >> 2) & 2))) << 5); }

// B operand (8 tokens of one column per lane) of column tile s from such a tile
__device__ __forceinline__ bf16x8 db_operand(const char* tile, int s, int lane) {
  const int row = 8 * (lane >> 4) + ((lane & 15) >> 2);
  const char* const p = tile + db_seg(row, s) + 8 * (lane & 3);
  const char* const p4 = tile + db_seg(row + 4, s) + 8 * (lane & 3);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p4));
  const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8, v);
}

// Token ranges for `groups` column groups of `steps` steps each: the number
// (at most `most`) for which the fullest CU has least to do, every range
// costing `extra` steps more (its first loads, its partials). The ranges of
// one CU share its issue, so what counts is how many it gets: 344 groups in 3
// ranges are 1032 workgroups, five of 43 steps on some of the 256 CUs, in 2
// ranges three of 64 (dB of 4096 x 22016, r = 64: 232 -> 217 us). One alone
// does not fill a CU and counts as two (dA of 4096 x 8192 from 256 workgroups
// 43 us, from 512 39).
inline int token_ranges(int64_t groups, int64_t steps, int64_t most, int64_t extra) {
  int best = 1;
  int64_t least = 0;
  for (int64_t s = 1; s <= most; ++s) {
    const int64_t share = cdiv(groups * s, (int64_t)256) > 2 ? cdiv(groups * s, (int64_t)256) : 2;
    const int64_t cost = share * (cdiv(steps, s) + extra);
    if (s == 1 || cost < least) {
      least = cost;
      best = (int)s;
    }
  }
  return best;
}

}  // namespace qlora
