// Pieces of the gradient kernels that contract over the tokens (gated.hip's
// dB, colgrad.hip): fp32 values in 16-bit parts, and the staged tile whose
// columns come back as MFMA operands.
#pragma once

#include "common.h"

namespace qlora {

// Eight fp32 values -> kParts 16-bit parts whose sum holds 24 (bf16, three)
// or 22 (fp16, two) bits of each.
template <bool kF16>
constexpr int parts_of() { return kF16 ? 2 : 3; }

template <bool kF16>
__device__ __forceinline__ void split8(const float (&x)[8], u32x4 (&p)[parts_of<kF16>()]) {
  float rem[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    rem[e] = x[e];
    // one fp32 value from here on: folded into the operation that made x, the
    // fp16 conversion stored and the one subtracted were rounded from
    // different values and a step apart for one element in 10^5
    asm("" : "+v"(rem[e]));
  }
#pragma unroll
  for (int q = 0; q < parts_of<kF16>(); ++q)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      p[q][w] = pack2<kF16>(rem[2 * w], rem[2 * w + 1]);
      asm("" : "+v"(p[q][w]));  // (unpacked from here, not converted a second time)
      rem[2 * w] -= from16<kF16>(p[q][w] & 0xFFFFu);
      rem[2 * w + 1] -= from16<kF16>(p[q][w] >> 16);
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
