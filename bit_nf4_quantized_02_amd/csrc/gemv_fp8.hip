// 8-bit layer for few tokens (M <= 16): one pass over the weight's codes.
//
//   Y = RN16( X8 W8^T + s T B^T ),   T = X A^T precomputed (fp32)
//
// Bound by HBM: every code byte serves at most 16 tokens. A first small
// kernel encodes X into the operand order of
// v_mfma_scale_f32_16x16x128_f8f6f4 (per 128-column block and lane: 32 bytes
// of one token row, zeros past M), so that the GEMV reads it in runs of 1 KB.
// A workgroup owns 16 kT weight rows; its 8 waves take the 128-column blocks
// in turn, so neighbouring waves read neighbouring lines of the same rows.
// Codes go from memory to registers in operand order (a lane holds 32
// consecutive bytes of one row, four lanes one 128-byte line), two batches of
// kU blocks rotating so that the next is in flight while one is multiplied.
// Partial sums of the waves are added in wave order through LDS, the low-rank
// term is added in fp32, and Y is rounded once.
#include "fp8.h"
#include "kernels.h"

namespace qlora {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kGvWaves = 8;
constexpr int kU = 2;  // 128-column blocks per batch

// One wave per 128-column block: lane (row lane % 16, columns 32 (lane / 16) ..)
template <bool kF16>
__global__ __launch_bounds__(256) void fp8_gemv_rows_kernel(const uint16_t* __restrict__ X, int64_t M, int64_t C,
                                                            int64_t nb, u32x4* __restrict__ Xq,
                                                            uint8_t* __restrict__ Xs) {
  const int lane = threadIdx.x & 63;
  const int64_t kb = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (kb >= nb) return;
  const int64_t m = lane & 15, c = kb * kF8Block + 32 * (lane >> 4);
  float f[32];
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (m < M && c < C) v = *reinterpret_cast<const u32x4*>(X + m * C + c + 8 * i);  // C % 64 == 0
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[8 * i + 2 * e] = from16<kF16>(v[e] & 0xFFFFu);
      f[8 * i + 2 * e + 1] = from16<kF16>(v[e] >> 16);
    }
  }
#pragma unroll
  for (int e = 0; e < 32; ++e) a = max(a, f8_finite_abs(f[e]));
  a = max(a, (uint32_t)__shfl_xor((int)a, 16));
  a = max(a, (uint32_t)__shfl_xor((int)a, 32));
  const uint32_t b = f8_scale_byte(a);
  const float inv = f8_inv_scale(b);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    Xq[(kb * 64 + lane) * 2 + h] = u32x4{f8_pack4(f + 16 * h, inv), f8_pack4(f + 16 * h + 4, inv),
                                         f8_pack4(f + 16 * h + 8, inv), f8_pack4(f + 16 * h + 12, inv)};
  if (lane < 16) Xs[kb * 16 + lane] = (uint8_t)b;
}

template <int kT>
struct Batch {
  u32x4 x[kU][2], w[kU][kT][2];
  uint32_t xs[kU], ws[kU];
};

__device__ __forceinline__ i32x8 join(const u32x4& lo, const u32x4& hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

template <int kT, bool kF16>
__global__ __launch_bounds__(64 * kGvWaves) void gemv_fp8_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ wscale, int64_t N,
                                                                 int64_t kp, const u32x4* __restrict__ Xq,
                                                                 const uint8_t* __restrict__ Xs, int64_t M,
                                                                 const float* __restrict__ T,
                                                                 const uint16_t* __restrict__ B, int r, float scale,
                                                                 uint16_t* __restrict__ Y) {
  constexpr int NT = 16 * kT;
  __shared__ float red[kGvWaves][kT][16][16];
  __shared__ float lred[kT][16][16];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * NT;
  const int nb = (int)(kp / kF8Block);
  const int64_t rows = N - n0 < NT ? N - n0 : NT;
  // this workgroup's rows (those past N read as zero and are not stored)
  const i32x4 wr = make_rsrc(codes + n0 * kp, rows * kp);
  const i32x4 sr = make_rsrc(wscale + (n0 / kF8Block) * nb, nb);
  // blocks past the end read as zero activations
  const i32x4 xr = make_rsrc(Xq, (int64_t)nb * 2048);
  const i32x4 xsr = make_rsrc(Xs, (int64_t)nb * 16);
  uint32_t woff[kT];
#pragma unroll
  for (int i = 0; i < kT; ++i) woff[i] = (uint32_t)((16 * i + (lane & 15)) * kp + 32 * (lane >> 4));

  auto load = [&](int j, Batch<kT>& b) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int kb = wave + kGvWaves * (j * kU + u);
      const int wb = kb < nb ? kb : nb - 1;
#pragma unroll
      for (int i = 0; i < kT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) b.w[u][i][h] = raw_buffer_load_b128(wr, (int)(woff[i] + 16 * h), wb * kF8Block, 0);
      b.ws[u] = raw_buffer_load_u8(sr, 0, wb, 0);
#pragma unroll
      for (int h = 0; h < 2; ++h) b.x[u][h] = raw_buffer_load_b128(xr, lane * 32 + 16 * h, kb * 2048, 0);
      b.xs[u] = raw_buffer_load_u8(xsr, lane & 15, kb * 16, 0);
    }
  };
  f32x4 acc[kT];
#pragma unroll
  for (int i = 0; i < kT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Batch<kT>& b) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < kT; ++i)
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(b.x[u][0], b.x[u][1]),
                                                                  join(b.w[u][i][0], b.w[u][i][1]), acc[i], 0, 0, 0,
                                                                  (int)b.xs[u], 0, (int)b.ws[u]);
  };
  const int cnt = (nb + kGvWaves * kU - 1) / (kGvWaves * kU);  // batches
  Batch<kT> b0, b1;
  load(0, b0);
  for (int j = 0; j < cnt; j += 2) {
    load(j + 1, b1);
    __builtin_amdgcn_sched_barrier(0);
    compute(b0);
    load(j + 2, b0);
    __builtin_amdgcn_sched_barrier(0);
    compute(b1);
  }

  // D[m][n]: lane -> n = lane % 16, m = 4 (lane / 16) + v
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) red[wave][i][4 * (lane >> 4) + v][lane & 15] = acc[i][v];
  if (r > 0 && wave < kT) {
    // L[m][n] = sum_j T[m][j] B[n][j], 4 ranks per fp32 MFMA (T and B exact)
    const int i = wave;
    f32x4 l = f32x4{0.f, 0.f, 0.f, 0.f};
    const int m = lane & 15;
    const int64_t n = n0 + i * 16 + (lane & 15);
    for (int j0 = 0; j0 < r; j0 += 4) {
      const int j = j0 + (lane >> 4);
      const float a = (m < M && j < r) ? T[m * r + j] : 0.0f;
      const float b = (n < N && j < r) ? from16<kF16>(B[n * r + j]) : 0.0f;
      l = __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, l, 0, 0, 0);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) lred[i][4 * (lane >> 4) + v][lane & 15] = l[v];
  }
  __syncthreads();
  for (int o = t; o < 16 * NT; o += 64 * kGvWaves) {
    const int m = o / NT, nl = o % NT;
    const int64_t n = n0 + nl;
    if (m >= M || n >= N) continue;
    const int i = nl >> 4, nc = nl & 15;
    float y = red[0][i][m][nc];
#pragma unroll
    for (int w = 1; w < kGvWaves; ++w) y += red[w][i][m][nc];  // in wave order
    if (r > 0) y = fmaf(scale, lred[i][m][nc], y);
    Y[m * N + n] = to16<kF16>(y);
  }
}

}  // namespace

size_t fp8_gemv_ws_bytes(int64_t k) {
  const int64_t nb = f8_pad(k) / kF8Block;
  return align256((size_t)nb * 2048) + align256((size_t)nb * 16);
}

hipError_t launch_fp8_gemv(const Fp8View& w, const uint16_t* X, int64_t M, const float* T, const uint16_t* B, int r,
                           float scale, uint16_t* Y, void* ws, hipStream_t stream, bool f16) {
  const int64_t kp = f8_pad(w.k), nb = kp / kF8Block;
  u32x4* const Xq = static_cast<u32x4*>(ws);
  uint8_t* const Xs = static_cast<uint8_t*>(ws) + align256((size_t)nb * 2048);
  const unsigned g0 = (unsigned)cdiv(nb, (int64_t)4);
  if (f16)
    fp8_gemv_rows_kernel<true><<<g0, 256, 0, stream>>>(X, M, w.k, nb, Xq, Xs);
  else
    fp8_gemv_rows_kernel<false><<<g0, 256, 0, stream>>>(X, M, w.k, nb, Xq, Xs);
#define QLORA_GV8(KT, H)                                                                                          \
  gemv_fp8_kernel<KT, H><<<(unsigned)cdiv(w.n, (int64_t)(16 * KT)), 64 * kGvWaves, 0, stream>>>(                   \
      w.codes, w.scale, w.n, kp, Xq, Xs, M, T, B, r, scale, Y)
  if (w.n >= 8192) {
    if (f16) QLORA_GV8(2, true); else QLORA_GV8(2, false);
  } else {
    if (f16) QLORA_GV8(1, true); else QLORA_GV8(1, false);
  }
#undef QLORA_GV8
  return hipGetLastError();
}

}  // namespace qlora
