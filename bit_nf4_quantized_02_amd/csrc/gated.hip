// Kernels of the gated feed-forward block around its two GEMMs (gemm_bf16.hip)
// and its few-token form (gemv_pair.hip):
//
//   G = X Wg'^T + s (X Ag^T) Bg^T,  U = X Wu'^T + s (X Au^T) Bu^T,  H = silu(G) U
//   dG = dH U sg (1 + G (1 - sg)),  dU = dH G sg,  sg = sigma(G)
//   dX = dG Wg' + dU Wu' + s (Pg Ag + Pu Au),  Pg = dG Bg, Pu = dU Bu
//   dAg = s Pg^T X,  dBg = s dG^T Tg,  and the same for u
//
// dG and dU enter dX's GEMM in 16 bits (its output has no more). The adapter
// gradients are fp32, so their products take the unrounded fp32 dG and dU as
// three bf16 parts, in fp16 too (colgrad.h). Neither G and U
// nor dG and dU are kept in fp32: the two kernels that need them compute them
// again from the 16-bit G, U and dH, which is fewer bytes than reading parts.
#include <type_traits>

#include "common.h"
#include "colgrad.h"
#include "fp8.h"
#include "gemm_tile.h"
#include "kernels.h"

namespace qlora {

namespace {

// ---------------------------------------------------------------- expansion

struct PairView {
  const uint32_t* codes;
  const uint8_t* code8;
  const float* s2;
  const float* mean;
  const float* codebook;
  const uint16_t* lr;  // B (forward) or A (dX)
};

constexpr int kRows = 8;  // weight rows per workgroup, as the plain row expansion

// One 16-byte output chunk column of 8 rows per thread; blockIdx.z picks the
// weight. kDx: rows stacked (weight z at rows z np .., zero rows from n to np)
// with pitch k; else interleaved in groups of 32 with the low-rank columns of
// the block's forward at the end of each row. Workgroups past the code chunks
// (blockIdx.y) write the low-rank columns, or for kDx (z == 2) the low-rank rows.
template <bool kDx, bool kF16>
__global__ __launch_bounds__(256) void gated_expand_kernel(PairView wg, PairView wu, bool s2_bf16, int64_t n, int64_t np,
                                                           int64_t k, int r, int xc, u32x4* __restrict__ out) {
  const int t = threadIdx.x, z = blockIdx.z;
  const int64_t kw = k / 8;
  const int64_t r0 = (int64_t)blockIdx.x * kRows;
  const int64_t c = (int64_t)blockIdx.y * 256 + t;
  if (kDx && z == 2) {
    // rows [Ag ; Ag ; Au ; Au ; 0] after the weights
    if (c >= kw) return;
    for (int i = 0; i < kRows; ++i) {
      const int64_t x = r0 + i;
      if (x >= xc) return;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (x < 4 * r) v = *reinterpret_cast<const u32x4*>((x < 2 * r ? wg.lr : wu.lr) + (x % r) * k + 8 * c);
      out[(2 * np + x) * kw + c] = v;
    }
    return;
  }
  const PairView w = z == 0 ? wg : wu;
  auto row_of = [&](int64_t i) -> int64_t { return kDx ? z * np + i : (i >> 5) * 64 + 32 * z + (i & 31); };
  const int64_t ldc = kDx ? kw : (k + xc) / 8;
  if (!kDx && (int64_t)blockIdx.y * 256 >= kw) {
    // columns [B | B] of this weight at 2r z, zero elsewhere
    const int cpr = xc / 8;
    for (int q = t; q < kRows * cpr; q += 256) {
      const int64_t i = r0 + q / cpr;
      if (i >= n) return;
      const int j0 = (q % cpr) * 8;
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = j0 + e - 2 * r * z;
        h[e] = j >= 0 && j < 2 * r ? (uint32_t)w.lr[i * r + (j < r ? j : j - r)] : 0u;
      }
      out[row_of(i) * ldc + kw + q % cpr] = u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                                                  h[6] | (h[7] << 16)};
    }
    return;
  }
  __shared__ float lut[16];
  if (t < 16) lut[t] = w.codebook[t];
  __syncthreads();
  if (c >= kw) return;
  const float mean = weight_mean(w.code8, w.mean);
  uint32_t word[kRows], c8[kRows];
  float s2v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t wi = (r0 + i < n ? r0 + i : n - 1) * kw + c;
    word[i] = w.codes[wi];
    scale_fields(w.code8, w.s2, s2_bf16, wi >> 3, c8[i], s2v[i]);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t row = r0 + i;
    if (row < n)
      out[row_of(row) * ldc + c] = dequant8<kF16>(word[i], lut, decode_block_scale(c8[i], s2v[i], mean));
    else if (kDx && row < np)
      out[row_of(row) * ldc + c] = u32x4{0u, 0u, 0u, 0u};
  }
}

// ------------------------------------------------------------------ the join

// sigma(g) from the hardware's 2^x and reciprocal (1 ulp each): the product -g
// log2 e carries half an ulp of itself into the exponent, 2^-24 |g| of sigma's
// tail, where sigma is small (13 instructions with both errors taken out
// against 4; the gradients' 2e-7 does not change). e^-g overflows to infinity
// for large negative g, where sigma is then 0, as it should be.
__device__ __forceinline__ float fast_sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g));
}

// dg = dh u (sg + silu (1 - sg)), du = dh silu, silu = g sg. In fp16 a finite G
// may have been saved as an infinity: silu is 0 at the lower one (not -inf 0),
// its derivative 0 and 1.
template <bool kF16>
__device__ __forceinline__ void join_bwd(float g, float u, float dh, float& dg, float& du) {
  const float sg = fast_sigmoid(g), rest = 1.0f - sg;
  float si = g * sg, bend = si;
  if constexpr (kF16) {
    if (sg == 0.0f) si = bend = 0.0f;
    if (rest == 0.0f) bend = 0.0f;
  }
  dg = dh * u * fmaf(bend, rest, sg);
  du = dh * si;
}

// dG and dU of eight adjacent elements.
template <bool kF16>
__device__ __forceinline__ void join8(const u32x4& g, const u32x4& u, const u32x4& dh, float (&dg)[8], float (&du)[8]) {
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      join_bwd<kF16>(from16<kF16>((g[w] >> (16 * h)) & 0xFFFFu), from16<kF16>((u[w] >> (16 * h)) & 0xFFFFu),
               from16<kF16>((dh[w] >> (16 * h)) & 0xFFFFu), dg[2 * w + h], du[2 * w + h]);
}

constexpr int kJoinWaves = 4;                // 16 rows each
constexpr int kJoinRows = 16 * kJoinWaves;

// A wave holds 16 rows and walks its workgroup's columns 64 at a time: eight
// neighbouring lanes load the 128 bytes of a row's line, dG and dU are formed
// in that layout and written rounded to D, and their parts pass one by one
// through the wave's own LDS into the A operand of v_mfma_f32_16x16x32 (lane:
// row lane % 16, columns 8 (lane / 16) ..). The step's factors, which the four
// waves share, are copied into LDS one step ahead. (Loaded straight in operand
// layout neighbouring lanes lie in different rows, 55 cache accesses per load:
// 340 us at 4096 x 22016, r = 64; in half lines, with the factors read by each
// wave: 276; so 208, 4.4 TB/s of the values read and written.) kRP: ranks padded (0: no adapters, D only).
// An fp16 B comes as its two bf16 parts; the third part of dG times the second
// of B is below the last bit kept.
template <int kRP, bool kF16, bool kVec>
__global__ __launch_bounds__(64 * kJoinWaves) void gated_join_kernel(
    const uint16_t* __restrict__ G, const uint16_t* __restrict__ U, const uint16_t* __restrict__ dH, int64_t M, int64_t n,
    int64_t np, const uint16_t* __restrict__ Bo, int r, int64_t cchunk, uint16_t* __restrict__ D,
    float* __restrict__ part) {
  constexpr int kTiles = kRP / 16, kTA = kTiles > 0 ? kTiles : 1;
  constexpr int kP = kParts, kB = parts16<kF16>();
  typedef typename std::conditional<kVec, u32x4, u32x4_any>::type Vec;
  // factors of a step: [w][32-column half][part][rank tile][1 KB], two steps in
  // two arrays (so that the compiler can tell the one being filled)
  __shared__ __attribute__((aligned(16))) char fac0[kTA * kB * 4096];
  __shared__ __attribute__((aligned(16))) char fac1[kTA * kB * 4096];
  // [wave][two buffers][16 rows x 128 bytes], 16-byte piece p of row i at p ^ (i / 2)
  __shared__ __attribute__((aligned(16))) char turn[kJoinWaves][2][kTiles > 0 ? 2048 : 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * kJoinRows + wave * 16;
  const int64_t cbeg = (int64_t)blockIdx.y * cchunk;
  const int64_t cend = cbeg + cchunk < np ? cbeg + cchunk : np;
  const int lr = lane >> 3, co = 8 * (lane & 7);  // loads: rows lr and lr + 8, columns co ..
  const int wr0 = lr * 128 + (((lane & 7) ^ (lr >> 1)) << 4), wr1 = (lr + 8) * 128 + (((lane & 7) ^ ((lr + 8) >> 1)) << 4);
  const int rrow = lane & 15;
  const int rd0 = rrow * 128 + (((lane >> 4) ^ (rrow >> 1)) << 4), rd1 = rrow * 128 + (((4 + (lane >> 4)) ^ (rrow >> 1)) << 4);
  int64_t off[2];  // row offsets (rows past M repeat the last one; not stored)
  bool in[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t m = m0 + 8 * u + lr;
    in[u] = m < M;
    off[u] = (m < M ? m : M - 1) * n + co;
  }
  f32x4 acc[2][kTA];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int t = 0; t < kTA; ++t) acc[w][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Stage {
    u32x4 g[2], u[2], d[2];
  };
  // whole steps load without a test per lane (a test would put each load behind
  // a branch that waits for it)
  auto load = [&](int64_t c, Stage& s) {
    if (c + 64 <= n) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        s.g[u] = *reinterpret_cast<const Vec*>(G + c + off[u]);
        s.u[u] = *reinterpret_cast<const Vec*>(U + c + off[u]);
        s.d[u] = *reinterpret_cast<const Vec*>(dH + c + off[u]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        s.g[u] = load8h<kVec>(G + off[u] - co, c + co, n);
        s.u[u] = load8h<kVec>(U + off[u] - co, c + co, n);
        s.d[u] = load8h<kVec>(dH + off[u] - co, c + co, n);
      }
    }
  };
  // this wave's share of a step's factors: weight wave / 2, half wave % 2
  constexpr int kFac = kB * kTiles;  // KB of 32 columns
  const i32x4 brs = make_rsrc(Bo + (wave >> 1) * (np / 32) * kFac * 512, np / 32 * kFac * 1024);
  auto copy_factors = [&](int64_t c, char* fac) {
    const uint32_t at = (uint32_t)(((c >> 5) + (wave & 1)) * kFac * 1024);
#pragma unroll
    for (int t = 0; t < kFac; ++t)
      copy16(brs, (uint32_t)lane * 16, (int)(at + t * 1024), fac + (wave * kFac + t) * 1024);
  };
  auto step = [&](int64_t c, const char* fac, char* next, Stage& cur, Stage& nxt) {
    // the factors of this step have landed, and every wave is done with the
    // buffer that the next ones go to (the six loads issued after them, or the
    // stores after those, may still be in flight)
    if constexpr (kTiles > 0) gt::step_barrier<4>();
    const int64_t cn = c + 64 < cend ? c + 64 : c;
    copy_factors(cn, next);
    __builtin_amdgcn_sched_barrier(0);  // (copies before loads: the next barrier's wait counts the operations after them)
    load(cn, nxt);
    __builtin_amdgcn_sched_barrier(0);
    float x[2][2][8];  // [row half][w]
#pragma unroll
    for (int u = 0; u < 2; ++u) join8<kF16>(cur.g[u], cur.u[u], cur.d[u], x[u][0], x[u][1]);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      u32x4 p[2][kP];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        split8(x[u][w], p[u]);
        u32x4 d = p[u][0];
        if constexpr (kF16) {
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = pack2<true>(x[u][w][2 * e], x[u][w][2 * e + 1]);
        }
        if (D != nullptr && in[u])
          *reinterpret_cast<u32x4*>(D + (m0 + 8 * u + lr) * 2 * np + w * np + c + co) = d;
      }
      if constexpr (kTiles > 0 && kF16) {
        bf16x8 a[kP][2];
#pragma unroll
        for (int q = 0; q < kP; ++q) {
          char* const buf = turn[wave][(w * kP + q) & 1];
          *reinterpret_cast<u32x4*>(buf + wr0) = p[0][q];
          *reinterpret_cast<u32x4*>(buf + wr1) = p[1][q];
          asm volatile("" ::: "memory");  // (as below)
          a[q][0] = *reinterpret_cast<const bf16x8*>(buf + rd0);
          a[q][1] = *reinterpret_cast<const bf16x8*>(buf + rd1);
          asm volatile("" ::: "memory");
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const char* const f = fac + lane * 16 + ((w * 2 + h) * kFac + t) * 1024;
            const bf16x8 hi = *reinterpret_cast<const bf16x8*>(f), lo = *reinterpret_cast<const bf16x8*>(f + kTiles * 1024);
#pragma unroll
            for (int q = kP - 1; q >= 0; --q) {
              if (q + 1 < kP) acc[w][t] = mfma16<false>(a[q][h], lo, acc[w][t]);
              acc[w][t] = mfma16<false>(a[q][h], hi, acc[w][t]);
            }
          }
      } else if constexpr (kTiles > 0) {
        bf16x8 b[2][kTA];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
            b[h][t] = *reinterpret_cast<const bf16x8*>(fac + lane * 16 + ((w * 2 + h) * kTiles + t) * 1024);
#pragma unroll
        for (int q = kP - 1; q >= 0; --q) {
          char* const buf = turn[wave][(w * kP + q) & 1];
          *reinterpret_cast<u32x4*>(buf + wr0) = p[0][q];
          *reinterpret_cast<u32x4*>(buf + wr1) = p[1][q];
          // lanes read what others wrote: the LDS keeps a wave's order, the
          // compiler must too
          asm volatile("" ::: "memory");
          const bf16x8 a0 = *reinterpret_cast<const bf16x8*>(buf + rd0), a1 = *reinterpret_cast<const bf16x8*>(buf + rd1);
          asm volatile("" ::: "memory");
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            acc[w][t] = mfma16<false>(a0, b[0][t], acc[w][t]);
            acc[w][t] = mfma16<false>(a1, b[1][t], acc[w][t]);
          }
        }
      }
    }
  };
  Stage s0, s1;
  copy_factors(cbeg, fac0);
  __builtin_amdgcn_sched_barrier(0);
  load(cbeg, s0);
  for (int64_t c = cbeg; c < cend; c += 128) {
    step(c, fac0, fac1, s0, s1);
    if (c + 64 < cend) step(c + 64, fac1, fac0, s1, s0);
  }
  // partials [split][w][M][r]; D layout: lane -> rank lane % 16, rows 4 (lane / 16) + v
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t m = m0 + 4 * (lane >> 4) + v;
        const int j = 16 * t + (lane & 15);
        if (m < M && j < r) part[(((int64_t)blockIdx.y * 2 + w) * M + m) * r + j] = acc[w][t][v];
      }
  // (copies of the repeated last step may still be landing: done before the workgroup's LDS is another's)
  __builtin_amdgcn_s_waitcnt(0);
}

// P = the partials added in split order; split row m = [hi_g | lo_g | hi_u |
// lo_u | 0] of scale P. One thread per (m, w, j), and for the padding columns.
__global__ __launch_bounds__(256) void gated_p_kernel(const float* __restrict__ part, int splits, int64_t M, int r,
                                                      int xc, float scale, float* __restrict__ P,
                                                      uint16_t* __restrict__ split) {
#pragma clang fp contract(off)
  const int per = xc - 2 * r;  // 2r products and xc - 4r zero columns
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (q >= M * per) return;
  const int64_t m = q / per;
  const int x = (int)(q % per);
  if (x >= 2 * r) {
    if (split) split[m * xc + 2 * r + x] = 0;
    return;
  }
  const int w = x >= r ? 1 : 0, j = x - w * r;
  // (eight loads together: those past the last repeat it and are not added)
  const float* const src = part + (w * M + m) * r + j;
  const int64_t pitch = 2 * M * r;
  float s = 0.0f;
  for (int p0 = 0; p0 < splits; p0 += 8) {
    float v[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) v[p] = src[(p0 + p < splits ? p0 + p : splits - 1) * pitch];
#pragma unroll
    for (int p = 0; p < 8; ++p)
      if (p0 + p < splits) s = p0 + p == 0 ? v[p] : s + v[p];
  }
  if (P) P[(w * M + m) * r + j] = s;
  if (split) {
    float v = scale * s;
    asm("" : "+v"(v));  // one value for both conversions (as split8)
    const uint16_t hi = to16<false>(v);
    split[m * xc + w * 2 * r + j] = hi;
    split[m * xc + w * 2 * r + r + j] = to16<false>(v - from16<false>(hi));
  }
}

// The fp16 form, of one or two factors (launch_scaled_columns): one row per
// wave, up to four of its W r values per lane.
__global__ __launch_bounds__(256) void scaled_columns_kernel(const float* __restrict__ part, int splits, int W, int64_t M,
                                                             int r, int xc, float scale, float* __restrict__ out,
                                                             uint16_t* __restrict__ split,
                                                             float* __restrict__ row_scale, bool apart) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x & 63;
  const int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= M) return;
  const int count = W * r;
  const int64_t pitch = (int64_t)W * M * r, pad = (M + 255) / 256 * 256;
  float v[4];
  uint32_t top[2] = {0, 0};  // of each factor
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = lane + 64 * e;
    v[e] = 0.0f;
    if (i >= count) continue;
    const int64_t at = ((int64_t)(i / r) * M + m) * r + i % r;
    float s = 0.0f;
    for (int p0 = 0; p0 < splits; p0 += 8) {
      float t[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) t[p] = part[at + (p0 + p < splits ? p0 + p : splits - 1) * pitch];
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (p0 + p < splits) s = p0 + p == 0 ? t[p] : s + t[p];
    }
    if (out) out[at] = s;
    v[e] = scale * s;
    asm("" : "+v"(v[e]));  // one value for the maximum and both conversions
    const uint32_t a = __float_as_uint(v[e]) & 0x7FFFFFFFu;
    top[0] = max(top[0], i < r ? a : 0u);
    top[1] = max(top[1], i < r ? 0u : a);
  }
  if (split == nullptr) return;
  if (!apart) top[0] = top[1] = max(top[0], top[1]);
  float down[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top[w] = max(top[w], (uint32_t)__shfl_xor((int)top[w], d));
    // largest value 1.x 2^(b - 127): e = b - 141, kept where 2^e and 2^-e are normal numbers
    // (a row with a value that is not finite, or of zeros, stays as it is)
    int e2 = (int)(top[w] >> 23) - 141;
    e2 = top[w] == 0 || top[w] >= 0x7F800000u ? 0 : e2 < -112 ? -112 : e2;
    down[w] = __uint_as_float((uint32_t)(127 - e2) << 23);
    if (lane == 0 && (w == 0 || apart)) row_scale[w * pad + m] = __uint_as_float((uint32_t)(127 + e2) << 23);
  }
  uint16_t* const row = split + m * xc;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = lane + 64 * e;
    if (i >= count) continue;
    float x = v[e] * (i < r ? down[0] : down[1]);
    asm("" : "+v"(x));
    const uint16_t hi = to16<true>(x);
    const int c = i / r * 2 * r + i % r;
    row[c] = hi;
    row[c + r] = to16<true>(x - from16<true>(hi));
  }
  for (int c = 2 * count + lane; c < xc; c += 64) row[c] = 0;
}

// ------------------------------------------------------ adapter gradients dB

// Partial of dB over tokens [m0, m1): rows = ranks, columns = block columns.
// Each 32-token step every thread forms dG and dU of one row's 8 columns and
// stages their parts as [token][column] tiles in LDS (two sets, one barrier
// per step); the B operand (8 tokens of one column per lane) comes back through
// the transposing read, the A operand (8 tokens of one rank) from Tt in runs.
// The four waves split the ranks first and then the columns, so that no rank
// row is loaded twice where there are at least 64. Products of parts whose
// order is below the last bit kept are left out (mid * lo and lo * lo). Bound by
// issue: forming and splitting dG and dU takes 54% of the cycles on the vector
// units, the products 35% on the matrix cores (4096 x 22016, r = 64: 215 us,
// where reading G, U and dH alone takes 108).
template <int kRP, bool kF16, bool kVec>
__global__ __launch_bounds__(256) void gated_db_kernel(const uint16_t* __restrict__ G, const uint16_t* __restrict__ U,
                                                       const uint16_t* __restrict__ dH, int64_t M, int64_t n,
                                                       const u32x4* __restrict__ Tt, int r, int64_t mchunk,
                                                       float* __restrict__ part) {
  constexpr int kP = kParts;
  constexpr int kJTall = kRP / 16;
  constexpr int kWJ = kJTall >= 4 ? 4 : kJTall;     // waves along ranks
  constexpr int kWC = 4 / kWJ;                      // waves along columns
  constexpr int kJT = kJTall / kWJ;                 // rank tiles per wave
  constexpr int kCT = kDbCols / 16 / kWC;           // column tiles per wave
  __shared__ __attribute__((aligned(16))) char sm[2 * 2 * kP * kDbTile];  // [set][w][part]
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wj = wave % kWJ, wc = wave / kWJ;
  const int64_t c0 = (int64_t)blockIdx.x * kDbCols;
  const int64_t m0 = (int64_t)blockIdx.y * mchunk;
  const int64_t m1 = m0 + mchunk < M ? m0 + mchunk : M;
  const int64_t pc = c0 + 8 * (t & 7);
  const int prow = t >> 3;
  struct Stage {
    u32x4 g, u, d;
  };
  const int64_t pcl = pc < n ? pc : n - 8;  // (columns past n repeat the last eight, their results are not stored)
  auto load = [&](int64_t mb, Stage& s) {
    const int64_t m = mb + prow;
    const int64_t o = (m < m1 ? m : m1 - 1) * n;
    if constexpr (kVec) {  // (no branch: behind one, the next wait for T's parts waits for these loads too)
      s.g = *reinterpret_cast<const u32x4*>(G + o + pcl);
      s.u = *reinterpret_cast<const u32x4*>(U + o + pcl);
      s.d = *reinterpret_cast<const u32x4*>(dH + o + pcl);
    } else if (c0 + kDbCols <= n) {
      s.g = *reinterpret_cast<const u32x4_any*>(G + o + pc);
      s.u = *reinterpret_cast<const u32x4_any*>(U + o + pc);
      s.d = *reinterpret_cast<const u32x4_any*>(dH + o + pc);
    } else {
      s.g = load8h<false>(G + o, pc, n);
      s.u = load8h<false>(U + o, pc, n);
      s.d = load8h<false>(dH + o, pc, n);
    }
  };
  // (rows past the range add nothing, whatever the row read in their place holds)
  auto stage = [&](int set, int64_t mb, Stage& s) {
    if (mb + 32 > m1 && mb + prow >= m1) s.g = s.u = s.d = u32x4{0u, 0u, 0u, 0u};
    float dg[8], du[8];
    join8<kF16>(s.g, s.u, s.d, dg, du);
    u32x4 p[kP];
    char* const at = sm + set * (2 * kP * kDbTile) + db_seg(prow, (t & 7) >> 1) + (t & 1) * 16;
    split8(dg, p);
#pragma unroll
    for (int q = 0; q < kP; ++q) *reinterpret_cast<u32x4*>(at + q * kDbTile) = p[q];
    split8(du, p);
#pragma unroll
    for (int q = 0; q < kP; ++q) *reinterpret_cast<u32x4*>(at + (kP + q) * kDbTile) = p[q];
  };
  f32x4 acc[2][kJT][kCT];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int a = 0; a < kJT; ++a)
#pragma unroll
      for (int b = 0; b < kCT; ++b) acc[w][a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  Stage st;
  if (m0 < m1) {
    load(m0, st);
    stage(0, m0, st);
    load(m0 + 32 < m1 ? m0 + 32 : m0, st);
  }
  __syncthreads();
  int set = 0;
  for (int64_t mb = m0; mb < m1; mb += 32, set ^= 1) {
    u32x4 ta[2][kP][kJT];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int q = 0; q < kP; ++q)
#pragma unroll
        for (int a = 0; a < kJT; ++a)
          ta[w][q][a] = Tt[((((mb >> 5) * kP + q) * 2 + w) * kJTall + wj * kJT + a) * 64 + lane];
    if (mb + 32 < m1) stage(set ^ 1, mb + 32, st);
    load(mb + 64 < m1 ? mb + 64 : m0, st);
    __builtin_amdgcn_sched_barrier(0);  // (issued here, not behind the products)
#pragma unroll
    for (int b = 0; b < kCT; ++b) {
      bf16x8 pb[2][kP];
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int q = 0; q < kP; ++q)
          pb[w][q] = db_operand(sm + ((set * 2 + w) * kP + q) * kDbTile, wc * kCT + b, lane);
#pragma unroll
      for (int order = kP - 1; order >= 0; --order)
#pragma unroll
        for (int q = 0; q <= order; ++q)
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int a = 0; a < kJT; ++a)
              acc[w][a][b] = mfma16<false>(__builtin_bit_cast(bf16x8, ta[w][order - q][a]), pb[w][q], acc[w][a][b]);
    }
    __syncthreads();
  }
  // D[j][c]: lane -> c = lane % 16, j = 4 (lane / 16) + v; partials [split][w][n][r], as dB
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int a = 0; a < kJT; ++a)
#pragma unroll
      for (int b = 0; b < kCT; ++b) {
        const int64_t c = c0 + 16 * (wc * kCT + b) + (lane & 15);
        const int j = 16 * (wj * kJT + a) + 4 * (lane >> 4);
        float* const o = part + (((int64_t)blockIdx.y * 2 + w) * n + c) * r + j;
        if (c < n && (r & 3) == 0 && j < r) {
          *reinterpret_cast<f32x4*>(o) = acc[w][a][b];
        } else if (c < n) {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (j + v < r) o[v] = acc[w][a][b][v];
        }
      }
}

// Column ranges of the join: about 1024 workgroups (each a multiple of 64
// columns; at most 32 ranges, whose partials are added later).
struct JoinPlan {
  int64_t cchunk;
  int splits;
};

JoinPlan join_plan(int64_t M, int64_t n) {
  const int64_t np = gated_pad(n);
  int64_t s = cdiv((int64_t)1024, cdiv(M, (int64_t)kJoinRows));
  if (s > np / 64) s = np / 64;
  if (s > 32) s = 32;
  const int64_t cchunk = cdiv(cdiv(np, s), (int64_t)64) * 64;
  return {cchunk, (int)cdiv(np, cchunk)};
}

// Token ranges of dB: each at least 128 tokens, at most 16.
struct DbPlan {
  int64_t mchunk;
  int splits;
};

DbPlan db_plan(int64_t M, int64_t n) {
  const int64_t steps = cdiv(M, (int64_t)32), most = cdiv(M, (int64_t)128);
  const int64_t s = token_ranges(cdiv(n, (int64_t)kDbCols), steps, most < 16 ? most : 16, 4);
  const int64_t mchunk = cdiv(steps, s) * 32;
  return {mchunk, (int)cdiv(M, mchunk)};
}

PairView pair_view(const Nf4View& w, const uint16_t* lr) {
  return PairView{reinterpret_cast<const uint32_t*>(w.codes), w.code8, w.s2, w.mean, w.codebook, lr};
}

}  // namespace

size_t gated_fwd_operand_bytes(int64_t n, int64_t k, int r) {
  return align256((size_t)gated_rows(n) * (size_t)(k + gated_extra_cols(r)) * 2);
}

hipError_t launch_gated_expand_fwd(const Nf4View& g, const Nf4View& u, const uint16_t* Bg, const uint16_t* Bu, int r,
                                   uint16_t* out, hipStream_t stream, bool f16) {
  const int xc = gated_extra_cols(r);
  const dim3 grid((unsigned)cdiv(g.n, (int64_t)kRows), (unsigned)(cdiv(g.k / 8, (int64_t)256) + (xc > 0 ? 1 : 0)), 2);
  u32x4* const o = reinterpret_cast<u32x4*>(out);
  const PairView a = pair_view(g, Bg), b = pair_view(u, Bu);
  if (f16)
    gated_expand_kernel<false, true><<<grid, 256, 0, stream>>>(a, b, g.s2_bf16, g.n, g.n, g.k, r, xc, o);
  else
    gated_expand_kernel<false, false><<<grid, 256, 0, stream>>>(a, b, g.s2_bf16, g.n, g.n, g.k, r, xc, o);
  return hipGetLastError();
}

size_t gated_dx_operand_bytes(int64_t n, int64_t k, int r) {
  return align256((size_t)(2 * gated_pad(n) + gated_extra_cols(r)) * (size_t)k * 2);
}

hipError_t launch_gated_expand_dx(const Nf4View& g, const Nf4View& u, const uint16_t* Ag, const uint16_t* Au, int r,
                                  uint16_t* out, hipStream_t stream, bool f16) {
  const int xc = gated_extra_cols(r);
  const int64_t np = gated_pad(g.n);
  const int64_t rows = np > xc ? np : xc;
  const dim3 grid((unsigned)cdiv(rows, (int64_t)kRows), (unsigned)cdiv(g.k / 8, (int64_t)256), xc > 0 ? 3 : 2);
  u32x4* const o = reinterpret_cast<u32x4*>(out);
  const PairView a = pair_view(g, Ag), b = pair_view(u, Au);
  if (f16)
    gated_expand_kernel<true, true><<<grid, 256, 0, stream>>>(a, b, g.s2_bf16, g.n, np, g.k, r, xc, o);
  else
    gated_expand_kernel<true, false><<<grid, 256, 0, stream>>>(a, b, g.s2_bf16, g.n, np, g.k, r, xc, o);
  return hipGetLastError();
}

namespace {

hipError_t launch_p(const float* part, int splits, int64_t M, int r, float scale, float* P, uint16_t* split,
                    float* row_scale, bool apart, hipStream_t stream, bool f16) {
  const int xc = gated_extra_cols(r);
  if (f16) return launch_scaled_columns(part, splits, 2, M, r, xc, scale, P, split, row_scale, stream, apart);
  const unsigned grid = (unsigned)cdiv(M * (xc - 2 * r), (int64_t)256);
  gated_p_kernel<<<grid, 256, 0, stream>>>(part, splits, M, r, xc, scale, P, split);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scaled_columns(const float* part, int splits, int W, int64_t M, int r, int xc, float scale, float* out,
                                 uint16_t* split, float* row_scale, hipStream_t stream, bool apart) {
  if (W < 1 || W > 2 || W * r > 256 || (split != nullptr && row_scale == nullptr)) return hipErrorInvalidValue;
  scaled_columns_kernel<<<(unsigned)cdiv(M, (int64_t)4), 256, 0, stream>>>(part, splits, W, M, r, xc, scale, out, split,
                                                                          row_scale, apart);
  return hipGetLastError();
}

size_t gated_project_ws_bytes(int64_t M, int64_t k, int r) {
  return align256(2 * operand_order_bytes(f8_pad(k), r)) +
         align256((size_t)fp8_prep_plan(M, k, false, 2).splits * 2 * M * r * 4);
}

hipError_t launch_gated_project(const uint16_t* X, int64_t M, int64_t k, const uint16_t* Ag, const uint16_t* Au, int r,
                                float scale, float* T, uint16_t* split, float* row_scale, void* ws, hipStream_t stream,
                                bool f16) {
  uint16_t* const Ao = static_cast<uint16_t*>(ws);
  float* const part = reinterpret_cast<float*>(static_cast<char*>(ws) + align256(2 * operand_order_bytes(f8_pad(k), r)));
  hipError_t e = launch_operand_order(Ag, Au, 0, k, f8_pad(k), r, Ao, stream);
  if (e == hipSuccess) e = launch_fp8_prep(X, M, k, Ao, r, nullptr, nullptr, part, false, stream, f16, 2);
  if (e == hipSuccess) e = launch_p(part, fp8_prep_plan(M, k, false, 2).splits, M, r, scale, T, split, row_scale,
                                    /*apart=*/true, stream, f16);
  return e;
}

// (B in operand order: both factors, an fp16 one in two parts)
size_t gated_join_ws_bytes(int64_t M, int64_t n, int r) {
  if (r == 0) return 0;
  return align256(4 * operand_order_bytes(gated_pad(n), r)) +
         align256((size_t)join_plan(M, n).splits * 2 * (size_t)M * r * 4);
}

hipError_t launch_gated_join(const uint16_t* G, const uint16_t* U, const uint16_t* dH, int64_t M, int64_t n,
                             const uint16_t* Bg, const uint16_t* Bu, int r, float scale, uint16_t* D, float* P,
                             uint16_t* split, float* row_scale, void* ws, hipStream_t stream, bool f16) {
  const JoinPlan pl = join_plan(M, n);
  const int64_t np = gated_pad(n);
  const int rp = rank_pad(r);
  uint16_t* const Bo = static_cast<uint16_t*>(ws);
  float* const part = reinterpret_cast<float*>(static_cast<char*>(ws) + align256(4 * operand_order_bytes(np, r)));
  if (r > 0) {
    const hipError_t e = launch_operand_order(Bg, Bu, 1, n, np, r, Bo, stream, f16);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)cdiv(M, (int64_t)kJoinRows), (unsigned)pl.splits);
#define QLORA_JOIN2(RP, H, V) \
  gated_join_kernel<RP, H, V><<<grid, 64 * kJoinWaves, 0, stream>>>(G, U, dH, M, n, np, Bo, r, pl.cchunk, D, part)
#define QLORA_JOIN(RP)                                                              \
  {                                                                                 \
    if (n % 8 == 0) { if (f16) QLORA_JOIN2(RP, true, true); else QLORA_JOIN2(RP, false, true); } \
    else { if (f16) QLORA_JOIN2(RP, true, false); else QLORA_JOIN2(RP, false, false); }          \
  }
  if (r == 0) QLORA_JOIN(0)
  else if (rp == 16) QLORA_JOIN(16)
  else if (rp == 32) QLORA_JOIN(32)
  else if (rp == 64) QLORA_JOIN(64)
  else QLORA_JOIN(128)
#undef QLORA_JOIN
#undef QLORA_JOIN2
  if (r > 0) return launch_p(part, pl.splits, M, r, scale, P, split, row_scale, /*apart=*/false, stream, f16);
  return hipGetLastError();
}

size_t gated_db_ws_bytes(int64_t M, int64_t n, int r) {
  if (r == 0) return 0;
  return align256((size_t)db_plan(M, n).splits * 2 * r * (size_t)n * 4);
}

hipError_t launch_gated_db(const uint16_t* G, const uint16_t* U, const uint16_t* dH, int64_t M, int64_t n,
                           const void* parts, int r, float* dBg, float* dBu, float* part, GradJob& job,
                           hipStream_t stream, bool f16) {
  const DbPlan pl = db_plan(M, n);
  const int rp = rank_pad(r);
  const u32x4* const Tt = static_cast<const u32x4*>(parts);
  job = GradJob{part, n * r, pl.splits, 2, dBg, dBu};
  const dim3 grid((unsigned)cdiv(n, (int64_t)kDbCols), (unsigned)pl.splits);
#define QLORA_DB2(RP, H, V) \
  gated_db_kernel<RP, H, V><<<grid, 256, 0, stream>>>(G, U, dH, M, n, Tt, r, pl.mchunk, part)
#define QLORA_DB(RP)                                                                         \
  {                                                                                          \
    if (n % 8 == 0) { if (f16) QLORA_DB2(RP, true, true); else QLORA_DB2(RP, false, true); }  \
    else { if (f16) QLORA_DB2(RP, true, false); else QLORA_DB2(RP, false, false); }           \
  }
  if (rp == 16) QLORA_DB(16)
  else if (rp == 32) QLORA_DB(32)
  else if (rp == 64) QLORA_DB(64)
  else QLORA_DB(128)
#undef QLORA_DB
#undef QLORA_DB2
  return hipGetLastError();
}

}  // namespace qlora
