// 8-bit layer for few tokens (M <= 16): one pass over the weight's codes.
//
//   Y = RN16( X8 W8^T + s T B^T )
//
// Bound by HBM: every code byte serves at most 16 tokens. fp8_prep_kernel has
// encoded X into the operand order of v_mfma_scale_f32_16x16x128_f8f6f4 (per
// 128-column block and lane: 32 bytes of one token row, zeros past M), so that
// X is read in runs of 1 KB, and left T = X A^T in a few partials, which each
// workgroup adds while its first codes are on the way (a launch less).
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
constexpr int kU = 2;      // 128-column blocks per batch
constexpr int kMaxR = 128;  // largest rank

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
                                                                 const float* __restrict__ T, int parts,
                                                                 const uint16_t* __restrict__ B, int r, float scale,
                                                                 uint16_t* __restrict__ Y, float* __restrict__ T_save) {
  constexpr int NT = 16 * kT;
  __shared__ float red[kGvWaves][kT][16][16];
  __shared__ float lred[kT][16][16];
  __shared__ float Ts[16 * kMaxR];  // T [M][r]
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
  for (int o = t; o < (int)M * r; o += 64 * kGvWaves) {
    float s = T[o];
    for (int p = 1; p < parts; ++p) s += T[(int64_t)p * M * r + o];
    Ts[o] = s;
    if (T_save != nullptr && blockIdx.x == 0) T_save[o] = s;
  }
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
  __syncthreads();  // T
  if (r > 0 && wave < kT) {
    // L[m][n] = sum_j T[m][j] B[n][j], 4 ranks per fp32 MFMA (T and B exact)
    const int i = wave;
    f32x4 l = f32x4{0.f, 0.f, 0.f, 0.f};
    const int m = lane & 15;
    const int64_t n = n0 + i * 16 + (lane & 15);
    for (int j0 = 0; j0 < r; j0 += 4) {
      const int j = j0 + (lane >> 4);
      const float a = (m < M && j < r) ? Ts[m * r + j] : 0.0f;
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

size_t fp8_gemv_codes_bytes(int64_t k) { return (size_t)(f8_pad(k) / kF8Block) * 2048; }
size_t fp8_gemv_scale_bytes(int64_t k) { return (size_t)(f8_pad(k) / kF8Block) * 16; }

hipError_t launch_fp8_gemv(const Fp8View& w, const uint8_t* xq, const uint8_t* xs, int64_t M, const float* T, int parts,
                           const uint16_t* B, int r, float scale, uint16_t* Y, float* T_save, hipStream_t stream,
                           bool f16) {
#define QLORA_GV8(KT, H)                                                                                          \
  gemv_fp8_kernel<KT, H><<<(unsigned)cdiv(w.n, (int64_t)(16 * KT)), 64 * kGvWaves, 0, stream>>>(                   \
      w.codes, w.scale, w.n, f8_pad(w.k), reinterpret_cast<const u32x4*>(xq), xs, M, T, parts, B, r, scale, Y, T_save)
  if (w.n >= 8192) {
    if (f16) QLORA_GV8(2, true); else QLORA_GV8(2, false);
  } else {
    if (f16) QLORA_GV8(1, true); else QLORA_GV8(1, false);
  }
#undef QLORA_GV8
  return hipGetLastError();
}

}  // namespace qlora
