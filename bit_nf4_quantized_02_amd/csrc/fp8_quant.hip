// Encoding into the 8-bit format and back (fp8.h): weights in 128 x 128
// tiles, activations in runs of 128 along a row. The kernels here are bound by
// HBM: one pass, every value read once and written once (22016 x 8192 from
// fp32: encode 173 us, 5.2 TB/s, decode 88).
#include <type_traits>

#include "fp8.h"
#include "gemm_tile.h"
#include "kernels.h"

namespace qlora {

namespace {

constexpr int kPrepRows = 128;  // activation rows per workgroup of fp8_prep_kernel

// 8 consecutive elements of a row as fp32, zero from element `lim` on.
// kDt: 0 bf16, 1 fp32, 2 fp16. kVec: 16-byte aligned rows.
template <int kDt, bool kVec>
__device__ __forceinline__ void load8f(const void* __restrict__ base, int64_t row_off, int64_t c, int64_t lim,
                                       float (&f)[8]) {
  if constexpr (kDt == 1) {
    const float* p = static_cast<const float*>(base) + row_off;
    if (kVec && c + 8 <= lim) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(p + c), b = *reinterpret_cast<const f32x4*>(p + c + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = a[i];
        f[4 + i] = b[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = c + i < lim ? p[c + i] : 0.0f;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + row_off;
    if (kVec && c + 8 <= lim) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(p + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = from16<kDt == 2>(v[i] & 0xFFFFu);
        f[2 * i + 1] = from16<kDt == 2>(v[i] >> 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = c + i < lim ? from16<kDt == 2>(p[c + i]) : 0.0f;
    }
  }
}

// One 128 x 128 weight tile per workgroup: thread t holds 8 columns of rows
// t / 16 + 16 i, so a tile is read once and stays in registers between the
// maximum and the rounding.
template <int kDt>
__global__ __launch_bounds__(256) void fp8_encode_kernel(const void* __restrict__ W, int64_t n, int64_t k, int64_t kp,
                                                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scale) {
  __shared__ uint32_t wmax[4];
  const int t = threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.y * kF8Block + (t >> 4), c = (int64_t)blockIdx.x * kF8Block + (t & 15) * 8;
  float f[8][8];
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    load8f<kDt, true>(W, (r < n ? r : n - 1) * k, c, k, f[i]);  // rows past n repeat the last one (not stored)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a = max(a, f8_finite_abs(f[i][e]));
      f[i][e] = isinf(f[i][e]) ? __uint_as_float(0x7FC00000u) : f[i][e];
    }
  }
  a = row16_max(a);
  a = max(a, (uint32_t)__shfl_xor((int)a, 16));
  a = max(a, (uint32_t)__shfl_xor((int)a, 32));
  if ((t & 63) == 0) wmax[t >> 6] = a;
  __syncthreads();
  a = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  const uint32_t b = f8_scale_byte(a);
  const float inv = f8_inv_scale(b);
  if (t == 0) scale[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = (uint8_t)b;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < n) *reinterpret_cast<u32x2*>(codes + r * kp + c) = u32x2{f8_pack4(f[i], inv), f8_pack4(f[i] + 4, inv)};
  }
}

// out = RN_bf16(value * scale): 16 codes per thread. Exact wherever bf16
// holds the product (all but the smallest scales).
__global__ __launch_bounds__(256) void fp8_decode_kernel(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scale, int64_t n, int64_t k,
                                                         int64_t kp, uint16_t* __restrict__ out) {
  const int64_t q = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  const int64_t per = k / 16;
  if (q >= n * per) return;
  const int64_t r = q / per, c = (q % per) * 16;
  const u32x4 v = *reinterpret_cast<const u32x4*>(codes + r * kp + c);
  const int e = (int)scale[(r / kF8Block) * (kp / kF8Block) + c / kF8Block] - 127;
  u32x4 o[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], true);
    o[i >> 1][2 * (i & 1)] = pack_bf16x2(ldexpf(lo[0], e), ldexpf(lo[1], e));
    o[i >> 1][2 * (i & 1) + 1] = pack_bf16x2(ldexpf(hi[0], e), ldexpf(hi[1], e));
  }
  u32x4* const p = reinterpret_cast<u32x4*>(out + r * k + c);
  p[0] = o[0];
  p[1] = o[1];
}

// Activations: one pass over P [M, C] that encodes it and forms its low-rank
// projection P Q^T (kRP ranks at most; 0: none) -- X with A in the forward, dY
// with B^T in the backward. A wave takes 128-column blocks of 16 rows: 16
// neighbouring lanes load one row's 256 bytes (8 columns each), find its
// maximum, and store its 128 code bytes; the values then pass through the
// wave's own LDS into the A operand of v_mfma_f32_16x16x32 (lane: row lane %
// 16, columns 8 (lane / 16) ..). Loaded in that layout straight from memory,
// neighbouring lanes lie in different rows and each of the 64 pieces is a
// cache access of its own, which was the kernel's bound (4096 x 22016, r = 64:
// 126 us).
//   kFew = false: codes [M, Cp] (zero past C) and the GEMM's scale words, one
// per (128-column block, 128-row tile, row % 32) with the bytes of rows +0,
// +32, +64, +96, so that a wave of the GEMM gets the scales of its four
// 32-row operand blocks with one load. A wave holds 32
// rows; the workgroup's four walk the blocks of one column range and share Q's,
// which are copied (in operand order) into LDS one block ahead.
//   kFew = true (M <= 16): codes in the GEMV's operand order [block][lane][32
// bytes] (lane: row lane % 16, bytes 32 (lane / 16) ..; zeros past M), scales
// [block][16]; Q [r, C] as it is. The four waves take the range's blocks in
// turn and their projections are added in wave order.
// Partials of the projection go to part [range][factor][M][r] (blockIdx.z: one of
// several factors, each over all of P); codes NULL: only those.
template <int kRP, bool kF16, bool kVec, bool kFew>
__global__ __launch_bounds__(256) void fp8_prep_kernel(const uint16_t* __restrict__ P, int64_t M, int64_t C, int64_t Cp,
                                                       const uint16_t* __restrict__ Q, int r, int bchunk,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scale,
                                                       float* __restrict__ part) {
  constexpr int kTiles = kRP / 16, kTA = kTiles > 0 ? kTiles : 1;
  constexpr int kMR = kFew ? 1 : 2;
  constexpr int kPitch = 256 + 16;  // bytes per staged row (16 rows on distinct banks)
  typedef typename std::conditional<kVec, u32x4, u32x4_any>::type Vec;
  __shared__ __attribute__((aligned(16))) char turn[4][kTiles > 0 ? 16 * kPitch : 16];
  // Q of a block, [32-column step][rank tile][1 KB], two blocks in two arrays
  // (so that the compiler can tell the one being filled)
  __shared__ __attribute__((aligned(16))) char fac0[kTiles > 0 && !kFew ? kTiles * 4096 : 16];
  __shared__ __attribute__((aligned(16))) char fac1[kTiles > 0 && !kFew ? kTiles * 4096 : 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = kFew ? 0 : (int64_t)blockIdx.x * kPrepRows + wave * 16 * kMR;
  const int64_t range = (int64_t)blockIdx.y * gridDim.z + blockIdx.z;  // partials: column range, then factor
  const int nb = (int)(Cp / kF8Block);
  const int b0 = (int)blockIdx.y * bchunk, b1 = b0 + bchunk < nb ? b0 + bchunk : nb;
  constexpr int kStep = kFew ? 4 : 1;
  const int64_t mt = cdiv(M, (int64_t)kF8Block);
  const int lr = lane >> 4, lc = 8 * (lane & 15);  // loads: row 4 u + lr, columns lc ..
  const uint16_t* prow[kMR][4];
#pragma unroll
  for (int i = 0; i < kMR; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t m = m0 + 16 * i + 4 * u + lr;
      prow[i][u] = P + (m < M ? m : M - 1) * C;
    }
  const uint16_t* qrow[kTA];  // kFew: this lane's rank rows
#pragma unroll
  for (int t = 0; t < kTiles; ++t) qrow[t] = Q + (kFew ? (int64_t)(16 * t + (lane & 15) < r ? 16 * t + (lane & 15) : r - 1) * C : 0);
  f32x4 acc[kMR][kTA];
#pragma unroll
  for (int i = 0; i < kMR; ++i)
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto load = [&](int kb, u32x4 (&x)[kMR][4]) {
    const int64_t c = (int64_t)kb * kF8Block + lc;
    if ((int64_t)(kb + 1) * kF8Block <= C) {  // (uniform: no load behind a test of its own)
#pragma unroll
      for (int i = 0; i < kMR; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) x[i][u] = *reinterpret_cast<const Vec*>(prow[i][u] + c);
    } else {
#pragma unroll
      for (int i = 0; i < kMR; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) x[i][u] = load8h<kVec>(prow[i][u], c, C);
    }
  };
  const i32x4 qrs = make_rsrc(Q + (int64_t)blockIdx.z * nb * kTiles * 2048, (int64_t)nb * kTiles * 4096);
  auto copy_q = [&](int kb, char* fac) {  // this wave's share: the block's 32-column step `wave`
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
      copy16(qrs, (uint32_t)lane * 16, (kb * 4 + wave) * kTiles * 1024 + t * 1024, fac + (wave * kTiles + t) * 1024);
  };
  auto block = [&](int kb, const char* fac, char* next, u32x4 (&x)[kMR][4], u32x4 (&nx)[kMR][4]) {
    const int kn = kb + kStep < b1 ? kb + kStep : kb;
    u32x4 q[kFew ? kTA : 1][4];
    if constexpr (kFew) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int64_t c = (int64_t)kb * kF8Block + 32 * s + 8 * (lane >> 4);
          q[t][s] = (int64_t)(kb + 1) * kF8Block <= C ? *reinterpret_cast<const u32x4*>(qrow[t] + c)
                                                      : load8h<true>(qrow[t], c, C);
        }
    } else if constexpr (kTiles > 0) {
      // this block's Q has landed, and every wave is done with the buffer the
      // next goes to (the eight loads issued after it, or stores after those,
      // may still be in flight)
      gt::step_barrier<4>();
      copy_q(kn, next);
      __builtin_amdgcn_sched_barrier(0);  // (copies before loads: the next barrier's wait counts the operations after them)
    }
    load(kn, nx);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kMR; ++i) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t m = m0 + 16 * i + 4 * u + lr;
        if (kFew && m >= M) x[i][u] = u32x4{0u, 0u, 0u, 0u};
        if constexpr (kTiles > 0)
          *reinterpret_cast<u32x4*>(turn[wave] + (4 * u + lr) * kPitch + 2 * lc) = x[i][u];
        if (codes != nullptr) {
          // the row's largest magnitude, from the 16-bit patterns (two at a
          // time, then the 16 lanes of the row by rotations within them)
          u16x2 top = {0, 0};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, x[i][u][e] & 0x7FFF7FFFu));
          uint32_t h = max((uint32_t)top[0], (uint32_t)top[1]);
          h = row16_max(h);
          float f[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[2 * e] = from16<kF16>(x[i][u][e] & 0xFFFFu);
            f[2 * e + 1] = from16<kF16>(x[i][u][e] >> 16);
          }
          if (__builtin_expect(__ballot(h >= (kF16 ? 0x7C00u : 0x7F80u)) != 0, 0)) {
            // a value of some row is not finite: the maximum without such values
            uint32_t a = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t v = f8_finite_abs(f[e]) != 0 ? (x[i][u][e >> 1] >> (16 * (e & 1))) & 0x7FFFu : 0u;
              a = max(a, v);
              if (isinf(f[e])) f[e] = __uint_as_float(0x7FC00000u);
            }
            h = row16_max(a);
          }
          const uint32_t b = f8_scale_byte(__float_as_uint(from16<kF16>(h)));
          const float inv = f8_inv_scale(b);
          const u32x2 o = {f8_pack4(f, inv), f8_pack4(f + 4, inv)};
          if constexpr (kFew) {
            // columns lc .. of row m: lane m + 16 (lc / 32), its bytes lc % 32 ..
            *reinterpret_cast<u32x2*>(codes + ((int64_t)kb * 64 + 16 * (lc >> 5) + 4 * u + lr) * 32 + (lc & 31)) = o;
            if ((lane & 15) == 0) scale[kb * 16 + 4 * u + lr] = (uint8_t)b;
          } else if (m < M) {
            *reinterpret_cast<u32x2*>(codes + m * Cp + (int64_t)kb * kF8Block + lc) = o;
            if ((lane & 15) == 0) scale[((kb * mt + m / kF8Block) * 32 + (m & 31)) * 4 + ((m >> 5) & 3)] = (uint8_t)b;
          }
        }
      }
      // lanes read what others wrote: the LDS keeps a wave's order, the
      // compiler must too
      asm volatile("" ::: "memory");
#pragma unroll
      for (int s = 0; s < (kTiles > 0 ? 4 : 0); ++s) {
        const bf16x8 pa = *reinterpret_cast<const bf16x8*>(turn[wave] + (lane & 15) * kPitch + 64 * s + 16 * (lane >> 4));
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if constexpr (kFew)
            acc[i][t] = mfma16<kF16>(pa, __builtin_bit_cast(bf16x8, q[t][s]), acc[i][t]);
          else
            acc[i][t] = mfma16<kF16>(pa, *reinterpret_cast<const bf16x8*>(fac + (s * kTiles + t) * 1024 + lane * 16), acc[i][t]);
        }
      }
      asm volatile("" ::: "memory");
    }
  };
  u32x4 x0[kMR][4], x1[kMR][4];
  const int kb0 = kFew ? b0 + wave : b0;
  if (kb0 < b1) {
    if constexpr (!kFew) copy_q(kb0, fac0);
    __builtin_amdgcn_sched_barrier(0);
    load(kb0, x0);
  }
  for (int kb = kb0; kb < b1; kb += 2 * kStep) {
    block(kb, fac0, fac1, x0, x1);
    if (kb + kStep < b1) block(kb + kStep, fac1, fac0, x1, x0);
  }
  // D layout: lane -> rank lane % 16, rows 4 (lane / 16) + v
  if constexpr (kRP > 0 && kFew) {
    __shared__ float red[4][16][kRP];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wave][4 * (lane >> 4) + v][16 * t + (lane & 15)] = acc[0][t][v];
    __syncthreads();
    for (int o = threadIdx.x; o < (int)M * r; o += 256) {
      const int m = o / r, j = o % r;
      part[(range * M + m) * r + j] = red[0][m][j] + red[1][m][j] + red[2][m][j] + red[3][m][j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kMR; ++i)
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t m = m0 + 16 * i + 4 * (lane >> 4) + v;
          const int j = 16 * t + (lane & 15);
          if (m < M && j < r) part[(range * M + m) * r + j] = acc[i][t][v];
        }
  }
  // (copies of the repeated last block may still be landing: done before the workgroup's LDS is another's)
  __builtin_amdgcn_s_waitcnt(0);
}

}  // namespace

hipError_t launch_fp8_encode(const void* W, int dt, int64_t n, int64_t k, uint8_t* codes, uint8_t* scale,
                             hipStream_t stream) {
  const int64_t kp = f8_pad(k);
  const dim3 grid((unsigned)(kp / kF8Block), (unsigned)cdiv(n, (int64_t)kF8Block));
  if (dt == QLORA_DT_FP32)
    fp8_encode_kernel<1><<<grid, 256, 0, stream>>>(W, n, k, kp, codes, scale);
  else if (dt == QLORA_DT_FP16)
    fp8_encode_kernel<2><<<grid, 256, 0, stream>>>(W, n, k, kp, codes, scale);
  else
    fp8_encode_kernel<0><<<grid, 256, 0, stream>>>(W, n, k, kp, codes, scale);
  return hipGetLastError();
}

hipError_t launch_fp8_decode(const Fp8View& w, uint16_t* out, hipStream_t stream) {
  // (a grid has less than 2^32 threads along one dimension: 2^36 elements at 16 each)
  const int64_t blocks = cdiv(w.n * (w.k / 16), (int64_t)256), y = cdiv(blocks, (int64_t)1 << 23);
  const dim3 grid((unsigned)cdiv(blocks, y), (unsigned)y);
  fp8_decode_kernel<<<grid, 256, 0, stream>>>(w.codes, w.scale, w.n, w.k, f8_pad(w.k), out);
  return hipGetLastError();
}

size_t fp8_rows_scale_bytes(int64_t M, int64_t C) {
  return (size_t)(f8_pad(C) / kF8Block) * (size_t)f8_pad(M);
}

// Column ranges: about 512 workgroups (1024 writes and reads twice the
// partials: 4096 x 22016, r = 64 93 against 84 us with the sum after it, 256
// 105), for two factors 512 in both together (512 each: 23 against 20 us at
// 2048 x 4096); at most 32 ranges. Few rows: one block per wave, at most 64
// ranges (the GEMV adds their partials).
Fp8Prep fp8_prep_plan(int64_t M, int64_t C, bool few, int W) {
  const int64_t nb = f8_pad(C) / kF8Block;
  int64_t s = few ? cdiv(nb, (int64_t)4) : cdiv((int64_t)(W == 1 ? 512 : 256), W * cdiv(M, (int64_t)kPrepRows));
  if (s > nb) s = nb;
  const int64_t most = few ? 64 : 32;
  if (s > most) s = most;
  const int64_t chunk = cdiv(nb, s);
  return Fp8Prep{(int)chunk, (int)cdiv(nb, chunk)};
}

hipError_t launch_fp8_prep(const uint16_t* P, int64_t M, int64_t C, const uint16_t* Q, int r,
                           uint8_t* codes, uint8_t* scale, float* part, bool few, hipStream_t stream, bool f16, int W) {
  const Fp8Prep pl = fp8_prep_plan(M, C, few, W);
  const int64_t Cp = f8_pad(C);
  if (few && (C % 8 != 0 || M > 16)) return hipErrorInvalidValue;
  if (W > 1 && (few || codes != nullptr)) return hipErrorInvalidValue;
  const dim3 grid(few ? 1u : (unsigned)cdiv(M, (int64_t)kPrepRows), (unsigned)pl.splits, (unsigned)W);
#define QLORA_PREP3(RP, H, V, F) \
  fp8_prep_kernel<RP, H, V, F><<<grid, 256, 0, stream>>>(P, M, C, Cp, Q, r, pl.chunk, codes, scale, part)
#define QLORA_PREP2(RP, H)                                                                             \
  {                                                                                                    \
    if (few) QLORA_PREP3(RP, H, true, true);                                                           \
    else if (C % 8 == 0) QLORA_PREP3(RP, H, true, false);                                              \
    else QLORA_PREP3(RP, H, false, false);                                                             \
  }
#define QLORA_PREP(RP) { if (f16) QLORA_PREP2(RP, true) else QLORA_PREP2(RP, false) }
  if (r == 0) QLORA_PREP(0)
  else if (r <= 16) QLORA_PREP(16)
  else if (r <= 32) QLORA_PREP(32)
  else if (r <= 64) QLORA_PREP(64)
  else QLORA_PREP(128)
#undef QLORA_PREP
#undef QLORA_PREP2
#undef QLORA_PREP3
  return hipGetLastError();
}

}  // namespace qlora
