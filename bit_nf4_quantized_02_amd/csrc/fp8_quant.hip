// Encoding into the 8-bit format and back (fp8.h): weights in 128 x 128
// tiles, activations in runs of 128 along a row. All four kernels here are
// bound by HBM: one pass, every value read once and written once.
#include "fp8.h"
#include "kernels.h"

namespace qlora {

namespace {

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
    for (int e = 0; e < 8; ++e) a = max(a, f8_finite_abs(f[i][e]));
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) a = max(a, (uint32_t)__shfl_xor((int)a, d));
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
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
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

// Activations X [M, C] -> codes [M, Cp] (zero past C) and scales for the GEMM:
// one 32-bit word per (128-column block, 128-row tile, row % 32) holding the
// bytes of rows +0, +32, +64, +96, so that a wave of the GEMM gets the scales
// of its four 32-row operand blocks with one load and picks each by the
// instruction's byte select. 16 threads per block of 128.
template <bool kF16, bool kVec>
__global__ __launch_bounds__(256) void fp8_rows_kernel(const uint16_t* __restrict__ X, int64_t M, int64_t C, int64_t Cp,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scale) {
  const int64_t u = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);  // (row, block)
  const int64_t nb = Cp / kF8Block;
  const int64_t m = u / nb, kb = u % nb;
  if (m >= M) return;
  const int64_t c = kb * kF8Block + (threadIdx.x & 15) * 8;
  float f[8];
  load8f<kF16 ? 2 : 0, kVec>(X, m * C, c, C, f);
  uint32_t a = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = max(a, f8_finite_abs(f[e]));
#pragma unroll
  for (int d = 1; d < 16; d *= 2) a = max(a, (uint32_t)__shfl_xor((int)a, d));
  const uint32_t b = f8_scale_byte(a);
  const float inv = f8_inv_scale(b);
  *reinterpret_cast<u32x2*>(codes + m * Cp + c) = u32x2{f8_pack4(f, inv), f8_pack4(f + 4, inv)};
  if ((threadIdx.x & 15) == 0) {
    const int64_t mt = cdiv(M, (int64_t)kF8Block);
    scale[((kb * mt + m / kF8Block) * 32 + (m & 31)) * 4 + ((m >> 5) & 3)] = (uint8_t)b;
  }
}

// Weight codes [n, kp] -> [k, np] (np: n up to a multiple of 128, zero past
// n), the operand whose rows run along dX's contraction. A thread turns 4
// rows x 16 columns in registers; 32 lanes write 128 contiguous bytes.
__global__ __launch_bounds__(256) void fp8_transpose_kernel(const uint8_t* __restrict__ codes, int64_t n, int64_t k,
                                                            int64_t kp, int64_t np, uint8_t* __restrict__ out) {
  const int64_t r0 = (int64_t)blockIdx.y * kF8Block + (threadIdx.x & 31) * 4;
  const int64_t c0 = (int64_t)blockIdx.x * kF8Block + (threadIdx.x >> 5) * 16;
  if (c0 >= k) return;
  u32x4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = *reinterpret_cast<const u32x4*>(codes + (r0 + i < n ? r0 + i : n - 1) * kp + c0);
    if (r0 + i >= n) v[i] = u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t sh = 8 * e;
      const uint32_t o = ((v[0][w] >> sh) & 0xFFu) | (((v[1][w] >> sh) & 0xFFu) << 8) |
                         (((v[2][w] >> sh) & 0xFFu) << 16) | (((v[3][w] >> sh) & 0xFFu) << 24);
      *reinterpret_cast<uint32_t*>(out + (c0 + 4 * w + e) * np + r0) = o;
    }
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
  const int64_t q = w.n * (w.k / 16);
  fp8_decode_kernel<<<(unsigned)cdiv(q, (int64_t)256), 256, 0, stream>>>(w.codes, w.scale, w.n, w.k, f8_pad(w.k), out);
  return hipGetLastError();
}

size_t fp8_rows_scale_bytes(int64_t M, int64_t C) {
  return (size_t)(f8_pad(C) / kF8Block) * (size_t)f8_pad(M);
}

hipError_t launch_fp8_rows(const uint16_t* X, int64_t M, int64_t C, uint8_t* codes, uint8_t* scale, hipStream_t stream,
                           bool f16) {
  const int64_t Cp = f8_pad(C);
  const unsigned grid = (unsigned)cdiv(M * (Cp / kF8Block), (int64_t)16);
#define QLORA_F8R(H, V) fp8_rows_kernel<H, V><<<grid, 256, 0, stream>>>(X, M, C, Cp, codes, scale)
  if (C % 8 == 0) {
    if (f16) QLORA_F8R(true, true); else QLORA_F8R(false, true);
  } else {
    if (f16) QLORA_F8R(true, false); else QLORA_F8R(false, false);
  }
#undef QLORA_F8R
  return hipGetLastError();
}

hipError_t launch_fp8_transpose(const Fp8View& w, uint8_t* out, hipStream_t stream) {
  const int64_t kp = f8_pad(w.k), np = f8_pad(w.n);
  const dim3 grid((unsigned)(kp / kF8Block), (unsigned)(np / kF8Block));
  fp8_transpose_kernel<<<grid, 256, 0, stream>>>(w.codes, w.n, w.k, kp, np, out);
  return hipGetLastError();
}

}  // namespace qlora
