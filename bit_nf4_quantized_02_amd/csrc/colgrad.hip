// Adapter gradients of the feed-forward operators: products over the tokens,
//
//   Gw[c, j] (+)= scale * sum_m P[m, c] Qw[m, j],   w = 0 (and 1, sharing P)
//
// P 16 bits [M, C], Qw fp32 [M, r]: dA = s P^T X from the fp32 projections, dB
// = s dY^T T. Q takes part with all its 24 bits, as three bf16 parts (an fp16 P
// as its two, exact): one small kernel writes Q's parts in operand order, and
// the products then read them in runs. Bound by HBM: P is read once for both Q.
// Against the layer calls' coldot kernel (lora.hip), which converts Q again in
// every workgroup and meets at two barriers per 32 tokens, a step here has one.
#include <type_traits>

#include "colgrad.h"
#include "kernels.h"

namespace qlora {

namespace {

constexpr int kMaxRank = 128;

// Q [W][M][r] -> [32-token step][part][w][rank tile][lane][16 bytes], the A
// operand of the products over the tokens: lane l holds rank 16 t + l % 16, tokens 8 (l / 16)
// .. +7 of the step, zero past M and r. Two such operands (of W0 and of the
// rest of gridDim.y) in one launch.
__global__ __launch_bounds__(256) void rank_parts_kernel(const float* __restrict__ Q0, int W0,
                                                         const float* __restrict__ Q1, int64_t M, int r, int tiles,
                                                         u32x4* __restrict__ out0, u32x4* __restrict__ out1) {
  __shared__ float tile[32][kMaxRank + 1];
  const bool first = (int)blockIdx.y < W0;
  const int w = first ? blockIdx.y : blockIdx.y - W0, W = first ? W0 : gridDim.y - W0;
  const float* const Q = first ? Q0 : Q1;
  u32x4* const out = first ? out0 : out1;
  const int64_t m0 = (int64_t)blockIdx.x * 32;
  // the step's 32 r values are one run (16-byte aligned): at most four loads per
  // thread, issued together
  const float* const src = Q + (w * M + m0) * r;
  const int64_t left = (M - m0) * r;
  const bool vec = ((uintptr_t)src & 15) == 0 && left >= 32 * r;
  if (vec) {
    f32x4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 4 * ((int)threadIdx.x + 256 * e);
      v[e] = *reinterpret_cast<const f32x4*>(src + (i < 32 * r ? i : 0));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = 4 * ((int)threadIdx.x + 256 * e) + x;
        if (i < 32 * r) tile[i / r][i % r] = v[e][x];
      }
  } else {
    for (int i = threadIdx.x; i < 32 * r; i += 256) tile[i / r][i % r] = i < left ? src[i] : 0.0f;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tiles * 64; i += 256) {
    const int j = 16 * (i >> 6) + (i & 15);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = j < r ? tile[8 * ((i >> 4) & 3) + e][j] : 0.0f;
    u32x4 p[kParts];
    split8(x, p);
#pragma unroll
    for (int q = 0; q < kParts; ++q) out[(((int64_t)blockIdx.x * kParts + q) * W + w) * tiles * 64 + i] = p[q];
  }
}

// A workgroup: 64 columns and one token range, 64 tokens per step in two sets of
// LDS (one barrier per step): every thread stages 16 bytes of two rows, the B
// operand (8 tokens of one column per lane) comes back through the transposing
// read, the A operand (8 tokens of one rank) from the parts in memory. The four
// waves split the ranks first and then the columns, so that no rank row is
// loaded twice where there are at least 64. kJFirst: results as [r, C] (else
// [C, r]); direct (one range): scaled and written, or added, to the gradient.
// (256 columns, which read the parts a quarter as often: 28 us against 18 for
// both factors over 2048 x 4096, r = 64, 44 against 40 over 4096 x 8192.)
template <int kRP, bool kF16, bool kVec, int kW, bool kJFirst>
__global__ __launch_bounds__(256) void colgrad_kernel(const uint16_t* __restrict__ P, int64_t M, int64_t C,
                                                      const u32x4* __restrict__ Qp, int r, int64_t mchunk,
                                                      float* __restrict__ part, bool direct, float scale,
                                                      float* __restrict__ G0, float* __restrict__ G1, int accumulate) {
  constexpr int kP = kParts, kX = parts16<kF16>();
  constexpr int kJTall = kRP / 16;
  constexpr int kWJ = kJTall >= 4 ? 4 : kJTall;  // waves along ranks
  constexpr int kWC = 4 / kWJ;                   // waves along columns
  constexpr int kJT = kJTall / kWJ;              // rank tiles per wave
  constexpr int kCT = kDbCols / 16 / kWC;        // column tiles per wave
  __shared__ __attribute__((aligned(16))) char sm[2 * 2 * kX * kDbTile];  // [set][32-token half][part of P]
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wj = wave % kWJ, wc = wave / kWJ;
  const int64_t c0 = (int64_t)blockIdx.x * kDbCols;
  const int64_t m0 = (int64_t)blockIdx.y * mchunk;
  const int64_t m1 = m0 + mchunk < M ? m0 + mchunk : M;
  const int prow = t >> 3;
  const int64_t pc = c0 + 8 * (t & 7);
  const int64_t pcl = pc < C ? pc : C - 8;  // (columns past C repeat the last eight, their results are not stored)
  struct Stage {
    u32x4 p[2];
  };
  auto load = [&](int64_t mb, Stage& s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t m = mb + 32 * h + prow;
      const uint16_t* const row = P + (m < m1 ? m : m1 - 1) * C;
      if constexpr (kVec)  // (no branch: behind one, the next wait for a part waits for this load too)
        s.p[h] = *reinterpret_cast<const u32x4*>(row + pcl);
      else
        s.p[h] = c0 + kDbCols <= C ? *reinterpret_cast<const u32x4_any*>(row + pc) : load8h<false>(row, pc, C);
    }
  };
  // (tokens past the range add nothing, whatever the row read in their place holds)
  auto stage = [&](int set, int64_t mb, Stage& s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (mb + 64 > m1 && mb + 32 * h + prow >= m1) s.p[h] = u32x4{0u, 0u, 0u, 0u};
      u32x4 x[kX];
      split8h<kF16>(s.p[h], x);
#pragma unroll
      for (int e = 0; e < kX; ++e)
        *reinterpret_cast<u32x4*>(sm + ((set * 2 + h) * kX + e) * kDbTile + db_seg(prow, (t & 7) >> 1) + (t & 1) * 16) = x[e];
    }
  };
  f32x4 acc[kW][kJT][kCT];
#pragma unroll
  for (int w = 0; w < kW; ++w)
#pragma unroll
    for (int a = 0; a < kJT; ++a)
#pragma unroll
      for (int b = 0; b < kCT; ++b) acc[w][a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  Stage st;
  if (m0 < m1) {
    load(m0, st);
    stage(0, m0, st);
    load(m0 + 64 < m1 ? m0 + 64 : m0, st);
  }
  __syncthreads();
  int set = 0;
  for (int64_t mb = m0; mb < m1; mb += 64, set ^= 1) {
    u32x4 q[2][kP][kW][kJT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // (the parts' rows end with the last token's 32: a half past it repeats that one against zeros)
      const int64_t ms = mb + 32 * h < m1 ? (mb >> 5) + h : (mb >> 5);
#pragma unroll
      for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int w = 0; w < kW; ++w)
#pragma unroll
          for (int a = 0; a < kJT; ++a)
            q[h][p][w][a] = Qp[(((ms * kP + p) * kW + w) * kJTall + wj * kJT + a) * 64 + lane];
    }
    if (mb + 64 < m1) stage(set ^ 1, mb + 64, st);
    load(mb + 128 < m1 ? mb + 128 : m0, st);
    __builtin_amdgcn_sched_barrier(0);  // (issued here, not behind the products)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < kCT; ++b) {
        bf16x8 pb[kX];
#pragma unroll
        for (int e = 0; e < kX; ++e) pb[e] = db_operand(sm + ((set * 2 + h) * kX + e) * kDbTile, wc * kCT + b, lane);
        // (the smallest products first; the third part of Q times the second of P is below the last bit kept)
#pragma unroll
        for (int p = kP - 1; p >= 0; --p)
#pragma unroll
          for (int e = kX - 1; e >= 0; --e)
#pragma unroll
            for (int w = 0; w < (p + e < kP ? kW : 0); ++w)
#pragma unroll
              for (int a = 0; a < kJT; ++a)
                acc[w][a][b] = mfma16<false>(__builtin_bit_cast(bf16x8, q[h][p][w][a]), pb[e], acc[w][a][b]);
      }
    __syncthreads();
  }
  // D[j][c]: lane -> c = lane % 16, j = 4 (lane / 16) + v
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    float* const G = direct ? (w == 0 ? G0 : G1) : part + ((int64_t)blockIdx.y * kW + w) * C * r;
    if (G == nullptr) continue;
#pragma unroll
    for (int a = 0; a < kJT; ++a)
#pragma unroll
      for (int b = 0; b < kCT; ++b) {
        const int64_t c = c0 + 16 * (wc * kCT + b) + (lane & 15);
        const int j = 16 * (wj * kJT + a) + 4 * (lane >> 4);
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (c < C && j + v < r) {
            float* const o = kJFirst ? G + (j + v) * C + c : G + c * r + j + v;
            const float x = acc[w][a][b][v];
            *o = !direct ? x : accumulate ? *o + scale * x : scale * x;
          }
      }
  }
}

// G (+)= scale * (partials [splits][W][count] added in order) of two jobs in
// one launch (blockIdx.z); a NULL gradient is left out. Four values per
// thread, whose first (a multiple of 4) is 16-byte aligned where count is.
__global__ __launch_bounds__(256) void grad_reduce_kernel(GradJob j0, GradJob j1, float scale, int accumulate) {
  const GradJob j = blockIdx.z == 0 ? j0 : j1;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int w = blockIdx.y;
  float* const G = w == 0 ? j.G0 : j.G1;
  if (i >= j.count || w >= j.W || G == nullptr) return;
  const float* const src = j.part + w * j.count + i;
  const int64_t pitch = (int64_t)j.W * j.count;
  if (j.count % 4 == 0) {
    f32x4 s = *reinterpret_cast<const f32x4*>(src);
#pragma unroll 4
    for (int p = 1; p < j.splits; ++p) s += *reinterpret_cast<const f32x4*>(src + p * pitch);
    f32x4* const o = reinterpret_cast<f32x4*>(G + i);
    s = scale * s;
    *o = accumulate ? *o + s : s;
  } else {
    for (int e = 0; e < 4 && i + e < j.count; ++e) {
      float s = src[e];
      for (int p = 1; p < j.splits; ++p) s += src[p * pitch + e];
      G[i + e] = accumulate ? G[i + e] + scale * s : scale * s;
    }
  }
}

// Token ranges: each at least 128 tokens, at most 16 (their partials are
// written and read again).
struct GradPlan {
  int64_t mchunk;
  int splits;
};

GradPlan grad_plan(int64_t M, int64_t C) {
  const int64_t steps = cdiv(M, (int64_t)64), most = cdiv(M, (int64_t)128);
  const int64_t s = token_ranges(cdiv(C, (int64_t)kDbCols), steps, most < 16 ? most : 16, 2);
  const int64_t mchunk = cdiv(steps, s) * 64;
  return {mchunk, (int)cdiv(M, mchunk)};
}

}  // namespace

size_t rank_parts_bytes(int64_t M, int r, int W) { return (size_t)cdiv(M, (int64_t)32) * kParts * W * rank_pad(r) * 64; }

hipError_t launch_rank_parts(const float* Q0, int W0, void* out0, const float* Q1, int W1, void* out1, int64_t M, int r,
                             hipStream_t stream) {
  const dim3 grid((unsigned)cdiv(M, (int64_t)32), (unsigned)(W0 + W1));
  u32x4 *const o0 = static_cast<u32x4*>(out0), *const o1 = static_cast<u32x4*>(out1);
  const int tiles = rank_pad(r) / 16;
  rank_parts_kernel<<<grid, 256, 0, stream>>>(Q0, W0, Q1, M, r, tiles, o0, o1);
  return hipGetLastError();
}

hipError_t launch_grad_reduce(const GradJob& a, const GradJob& b, float scale, int accumulate, hipStream_t stream) {
  if (a.W == 0 && b.W == 0) return hipSuccess;
  const int64_t count = a.count > b.count ? a.count : b.count;
  const dim3 grid((unsigned)cdiv(count, (int64_t)1024), (unsigned)(a.W > b.W ? a.W : b.W), 2);
  grad_reduce_kernel<<<grid, 256, 0, stream>>>(a, b, scale, accumulate);
  return hipGetLastError();
}

size_t colgrad_ws_bytes(int64_t M, int64_t C, int r, int W) {
  const GradPlan pl = grad_plan(M, C);
  return pl.splits > 1 ? align256((size_t)pl.splits * W * r * (size_t)C * 4) : 0;
}

hipError_t launch_colgrad(const uint16_t* P, int64_t M, int64_t C, const void* parts, int W, int r, float scale,
                          float* G0, float* G1, bool j_first, int accumulate, float* part, GradJob& job,
                          hipStream_t stream, bool f16) {
  const u32x4* const Qp = static_cast<const u32x4*>(parts);
  const GradPlan pl = grad_plan(M, C);
  const bool direct = pl.splits == 1;
  job = GradJob{};
  if (!direct) job = GradJob{part, C * r, pl.splits, W, G0, G1};
  const dim3 grid((unsigned)cdiv(C, (int64_t)kDbCols), (unsigned)pl.splits);
#define QLORA_CG3(RP, H, V, NW, J) \
  colgrad_kernel<RP, H, V, NW, J><<<grid, 256, 0, stream>>>(P, M, C, Qp, r, pl.mchunk, part, direct, scale, G0, G1, accumulate)
// (X's gradients are [r, k] with k a multiple of 64, of one adapter or two; dY's are [n, r])
#define QLORA_CG2(RP, H)                                                                                     \
  {                                                                                                          \
    if (j_first) { if (W == 2) QLORA_CG3(RP, H, true, 2, true); else QLORA_CG3(RP, H, true, 1, true); }       \
    else if (C % 8 == 0) QLORA_CG3(RP, H, true, 1, false);                                                   \
    else QLORA_CG3(RP, H, false, 1, false);                                                                  \
  }
#define QLORA_CG(RP) { if (f16) QLORA_CG2(RP, true) else QLORA_CG2(RP, false) }
  if (j_first ? C % 8 != 0 : W != 1) return hipErrorInvalidValue;
  if (r <= 16) QLORA_CG(16)
  else if (r <= 32) QLORA_CG(32)
  else if (r <= 64) QLORA_CG(64)
  else QLORA_CG(128)
#undef QLORA_CG
#undef QLORA_CG2
#undef QLORA_CG3
  return hipGetLastError();
}

}  // namespace qlora
