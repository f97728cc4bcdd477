// Residual addition with the root-mean-square norm, and its backward.
//
//   h = RN16(RN32(x + res)),  rstd = (mean(h^2) + eps)^-1/2,  y = RN16(h rstd w)
//   g = dy w,  hn = h rstd,  dx = RN16(rstd (g - hn mean(g hn)) + dres),  dw = sum over rows of dy hn
//
// Sums and rstd are fp32. The stream h is rounded before it is normalised: the
// backward, which reads it again, then differentiates what was computed. As 8-bit
// activations (fp8.h) the 16-bit y is encoded, so that the layer gets the same
// codes from here as it makes of y itself.
//
// Bound by HBM: every value is read once and stays in registers between the sum
// and its use. kLpr lanes hold a row, kV runs of 8 values each; 16 neighbouring
// lanes hold 128 columns, a scale block of the 8-bit form. Rows of more than 32768
// columns do not fit a workgroup's registers and are read twice.
#include "fp8.h"
#include "kernels.h"

namespace qlora {

namespace {

constexpr int64_t kInRegisters = 32768;  // columns of a row that a workgroup holds

// Eight 16-bit values into (row, c), nothing from n on.
template <bool kVec>
__device__ __forceinline__ void store8h(uint16_t* __restrict__ row, int64_t c, int64_t n, const u32x4& v) {
  if constexpr (kVec) {
    if (c < n) *reinterpret_cast<u32x4*>(row + c) = v;
  } else if (c + 8 <= n) {
    *reinterpret_cast<u32x4_any*>(row + c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
  }
}

// Eight gains from c on, as they are stored: 16 bits in a[0], or fp32.
struct Gain {
  u32x4 a[2];
};

template <bool kVec>
__device__ __forceinline__ Gain load_gain(const void* __restrict__ w, bool w32, int64_t c, int64_t n) {
  Gain g;
  if (!w32) {
    g.a[0] = load8h<kVec>(static_cast<const uint16_t*>(w), c, n);
    g.a[1] = u32x4{0u, 0u, 0u, 0u};
    return g;
  }
  const uint32_t* p = static_cast<const uint32_t*>(w);
  if (c + 8 <= n) {
    g.a[0] = *reinterpret_cast<const u32x4*>(p + c);
    g.a[1] = *reinterpret_cast<const u32x4*>(p + c + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t e = p[c + i < n ? c + i : n - 1];
      g.a[i >> 2][i & 3] = c + i < n ? e : 0u;
    }
  }
  return g;
}

template <bool kF16>
__device__ __forceinline__ void gain8(const Gain& g, bool w32, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = from16<kF16>((g.a[0][i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
    f[i] = w32 ? __uint_as_float(g.a[i >> 2][i & 3]) : s;
  }
}

template <bool kF16>
__device__ __forceinline__ void unpack8(const u32x4& v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = from16<kF16>((v[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
}

template <bool kF16>
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{pack2<kF16>(f[0], f[1]), pack2<kF16>(f[2], f[3]), pack2<kF16>(f[4], f[5]), pack2<kF16>(f[6], f[7])};
}

template <int kCtrl>
__device__ __forceinline__ float rotated(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), kCtrl, 0xF, 0xF, true));
}

// Sum over the kLpr lanes of a row, in all of them and in one order always.
// red: one float for each wave of the workgroup, used when a row has more than
// one wave (then every thread of the workgroup calls).
template <int kLpr>
__device__ __forceinline__ float row_sum(float s, float* red) {
  s += rotated<0x128>(s);
  s += rotated<0x124>(s);
  s += rotated<0x122>(s);
  s += rotated<0x121>(s);
  if constexpr (kLpr >= 64) {
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
  }
  if constexpr (kLpr > 64) {
    constexpr int kWaves = kLpr / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) s += red[wave / kWaves * kWaves + i];
  }
  return s;
}

// h from X and the residual (16-bit patterns of eight values).
template <bool kF16>
__device__ __forceinline__ u32x4 add8(const u32x4& x, const u32x4& r) {
  float a[8], b[8];
  unpack8<kF16>(x, a);
  unpack8<kF16>(r, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] += b[i];
  return pack8<kF16>(a);
}

template <bool kF16>
__device__ __forceinline__ float squares8(const u32x4& h, float s) {
  float f[8];
  unpack8<kF16>(h, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
  return s;
}

// y of eight values, in 16 bits.
template <bool kF16>
__device__ __forceinline__ u32x4 normed8(const u32x4& h, float rstd, const Gain& g, bool w32) {
  float f[8], w[8];
  unpack8<kF16>(h, f);
  gain8<kF16>(g, w32, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = f[i] * rstd * w[i];
  return pack8<kF16>(f);
}

// The 8-bit form of y: 16 neighbouring lanes (all of them call) hold a block of
// 128 columns and find its scale; columns c .. of row m are this lane's.
template <bool kF16>
__device__ __forceinline__ void encode8(const u32x4& y, int64_t m, int64_t c, int64_t kp, uint8_t* __restrict__ codes,
                                        uint8_t* __restrict__ scale) {
  u16x2 top = {0, 0};
#pragma unroll
  for (int e = 0; e < 4; ++e) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, y[e] & 0x7FFF7FFFu));
  uint32_t h = row16_max(max((uint32_t)top[0], (uint32_t)top[1]));
  float f[8];
  unpack8<kF16>(y, f);
  if (__builtin_expect(__ballot(h >= (kF16 ? 0x7C00u : 0x7F80u)) != 0, 0)) {
    // a value of some row is not finite: the maximum without such values
    uint32_t a = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a = max(a, f8_finite_abs(f[e]) != 0 ? (y[e >> 1] >> (16 * (e & 1))) & 0x7FFFu : 0u);
      if (isinf(f[e])) f[e] = __uint_as_float(0x7FC00000u);
    }
    h = row16_max(a);
  }
  const uint32_t b = f8_scale_byte(__float_as_uint(from16<kF16>(h)));
  const float inv = f8_inv_scale(b);
  *reinterpret_cast<u32x2*>(codes + m * kp + c) = u32x2{f8_pack4(f, inv), f8_pack4(f + 4, inv)};
  if ((c & (kF8Block - 1)) == 0) scale[m * (kp / kF8Block) + c / kF8Block] = (uint8_t)b;
}

struct FwdArgs {
  const uint16_t *X, *R;  // R: the residual, or NULL
  const void* w;
  int w32;
  int64_t M, k, kp;
  float inv_k, eps;
  uint16_t *Y, *H;        // Y may be NULL; H is there if R is
  float* rstd;            // may be NULL
  uint8_t *codes, *scale; // may be NULL
};

template <bool kF16, int kLpr, int kV, bool kVec>
__global__ __launch_bounds__(kLpr < 256 ? 256 : kLpr) void rms_fwd_kernel(FwdArgs a) {
  constexpr int kThreads = kLpr < 256 ? 256 : kLpr;
  __shared__ float red[kThreads / 64];
  const int t = threadIdx.x & (kLpr - 1);
  const int64_t m = (int64_t)blockIdx.x * (kThreads / kLpr) + threadIdx.x / kLpr;
  const bool live = m < a.M;
  const int64_t at = (live ? m : a.M - 1) * a.k;
  u32x4 h[kV], r[kV];
  Gain g[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) h[v] = load8h<kVec>(a.X + at, 8 * (t + kLpr * v), a.k);
  if (a.R != nullptr) {
#pragma unroll
    for (int v = 0; v < kV; ++v) r[v] = load8h<kVec>(a.R + at, 8 * (t + kLpr * v), a.k);
  }
#pragma unroll
  for (int v = 0; v < kV; ++v) g[v] = load_gain<kVec>(a.w, a.w32, 8 * (t + kLpr * v), a.k);
  if (a.R != nullptr) {
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      h[v] = add8<kF16>(h[v], r[v]);
      if (live) store8h<kVec>(a.H + at, 8 * (t + kLpr * v), a.k, h[v]);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < kV; ++v) s = squares8<kF16>(h[v], s);
  const float rstd = 1.0f / sqrtf(fmaf(row_sum<kLpr>(s, red), a.inv_k, a.eps));
  if (!live) return;
  if (t == 0 && a.rstd != nullptr) a.rstd[m] = rstd;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int64_t c = 8 * (t + kLpr * v);
    const u32x4 y = normed8<kF16>(h[v], rstd, g[v], a.w32);
    if (a.Y != nullptr) store8h<kVec>(a.Y + at, c, a.k, y);
    if (kVec && a.codes != nullptr && c < a.kp) encode8<kF16>(y, m, c, a.kp, a.codes, a.scale);
  }
}

// Rows of any length, read twice (the second time from the caches, if they hold
// a row of every workgroup).
template <bool kF16, bool kVec>
__global__ __launch_bounds__(1024) void rms_fwd_long_kernel(FwdArgs a) {
  __shared__ float red[16];
  const int64_t m = blockIdx.x, at = m * a.k;
  const uint16_t* const in = a.R != nullptr ? a.H + at : a.X + at;
  float s = 0.0f;
  for (int64_t c = 8 * threadIdx.x; c < a.k; c += 8192) {
    u32x4 h = load8h<kVec>(a.X + at, c, a.k);
    if (a.R != nullptr) {
      h = add8<kF16>(h, load8h<kVec>(a.R + at, c, a.k));
      store8h<kVec>(a.H + at, c, a.k, h);
    }
    s = squares8<kF16>(h, s);
  }
  const float rstd = 1.0f / sqrtf(fmaf(row_sum<1024>(s, red), a.inv_k, a.eps));
  if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[m] = rstd;
  for (int64_t c = 8 * threadIdx.x; c < a.kp; c += 8192) {  // (each thread reads what it wrote)
    const u32x4 y = normed8<kF16>(load8h<kVec>(in, c, a.k), rstd, load_gain<kVec>(a.w, a.w32, c, a.k), a.w32);
    if (a.Y != nullptr) store8h<kVec>(a.Y + at, c, a.k, y);
    if (kVec && a.codes != nullptr) encode8<kF16>(y, m, c, a.kp, a.codes, a.scale);
  }
}

struct BwdArgs {
  const uint16_t *dY, *H, *R;  // R: the gradient that reaches h past the norm, or NULL
  const float* rstd;
  const void* w;
  int w32;
  int64_t M, k;
  float inv_k;
  uint16_t* dX;  // may be NULL
  float* part;   // kDw: partial sums of dw, [workgroup][k]
};

// dx of eight values; dot: mean(g hn)
template <bool kF16>
__device__ __forceinline__ u32x4 dx8(const u32x4& dy, const u32x4& h, const u32x4& r, bool has_r, float rstd, float dot,
                                     const float (&w)[8]) {
  float a[8], b[8], d[8];
  unpack8<kF16>(dy, a);
  unpack8<kF16>(h, b);
  unpack8<kF16>(r, d);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = rstd * (a[i] * w[i] - b[i] * rstd * dot);
    a[i] = has_r ? x + d[i] : x;
  }
  return pack8<kF16>(a);
}

// Workgroups of kThreads hold kThreads / kLpr rows at a time and walk over the
// rows with the grid. kDw: each lane adds up dy hn of its columns over the
// rows it meets; the rows of a workgroup are joined in LDS at the end, the
// workgroups by rms_dw_kernel.
template <bool kF16, int kLpr, int kV, int kThreads, bool kVec, bool kDw>
__global__ __launch_bounds__(kThreads) void rms_bwd_kernel(BwdArgs a) {
  constexpr int kRows = kThreads / kLpr;
  __shared__ float red[2][kThreads / 64];
  const int t = threadIdx.x & (kLpr - 1), group = threadIdx.x / kLpr;
  float w[kV][8], acc[kV][8];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const Gain g = load_gain<kVec>(a.w, a.w32, 8 * (t + kLpr * v), a.k);
    gain8<kF16>(g, a.w32, w[v]);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.0f;
  }
  struct Row {
    u32x4 dy[kV], h[kV], r[kV];
    float rstd;
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  auto load = [&](int64_t m0, Row& x) {
    const int64_t m = m0 + group < a.M ? m0 + group : a.M - 1;
    const int64_t at = m * a.k;
    x.rstd = a.rstd[m];
#pragma unroll
    for (int v = 0; v < kV; ++v) x.dy[v] = load8h<kVec>(a.dY + at, 8 * (t + kLpr * v), a.k);
#pragma unroll
    for (int v = 0; v < kV; ++v) x.h[v] = load8h<kVec>(a.H + at, 8 * (t + kLpr * v), a.k);
#pragma unroll
    for (int v = 0; v < kV; ++v)
      x.r[v] = a.R != nullptr ? load8h<kVec>(a.R + at, 8 * (t + kLpr * v), a.k) : u32x4{0u, 0u, 0u, 0u};
  };
  int turn = 0;
  auto row = [&](int64_t m0, const Row& x) {
    const bool live = m0 + group < a.M;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      float dy[8], h[8];
      unpack8<kF16>(x.dy[v], dy);
      unpack8<kF16>(x.h[v], h);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = dy[i] * (h[i] * x.rstd);
        s = fmaf(p, w[v][i], s);
        if (kDw && live) acc[v][i] += p;
      }
    }
    // (two buffers in turn: one barrier a row)
    const float dot = row_sum<kLpr>(s, red[turn]) * a.inv_k;
    turn ^= 1;
    if (!live || a.dX == nullptr) return;
#pragma unroll
    for (int v = 0; v < kV; ++v)
      store8h<kVec>(a.dX + (m0 + group) * a.k, 8 * (t + kLpr * v), a.k,
                    dx8<kF16>(x.dy[v], x.h[v], x.r[v], a.R != nullptr, x.rstd, dot, w[v]));
  };
  Row x0, x1;
  int64_t m0 = (int64_t)blockIdx.x * kRows;
  load(m0, x0);
  for (; m0 < a.M; m0 += 2 * step) {
    if (m0 + step < a.M) load(m0 + step, x1);
    row(m0, x0);
    if (m0 + step >= a.M) break;
    if (m0 + 2 * step < a.M) load(m0 + 2 * step, x0);
    row(m0 + step, x1);
  }
  if constexpr (kDw) {
    constexpr int kCols = 8 * kLpr * kV;
    float* const out = a.part + (int64_t)blockIdx.x * a.k;
    if constexpr (kRows == 1) {
#pragma unroll
      for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t c = 8 * (t + kLpr * v) + i;
          if (c < a.k) out[c] = acc[v][i];
        }
    } else {
      __shared__ float join[kRows][kCols];
#pragma unroll
      for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) join[group][8 * (t + kLpr * v) + i] = acc[v][i];
      __syncthreads();
      for (int c = threadIdx.x; c < kCols && c < a.k; c += kThreads) {
        float s = join[0][c];
#pragma unroll 8
        for (int g = 1; g < kRows; ++g) s += join[g][c];
        out[c] = s;
      }
    }
  }
}

// dX for rows of any length, one workgroup a row, which is read twice.
template <bool kF16, bool kVec>
__global__ __launch_bounds__(1024) void rms_bwd_long_kernel(BwdArgs a) {
  __shared__ float red[16];
  const int64_t at = (int64_t)blockIdx.x * a.k;
  const float rstd = a.rstd[blockIdx.x];
  float s = 0.0f;
  for (int64_t c = 8 * threadIdx.x; c < a.k; c += 8192) {
    float dy[8], h[8], w[8];
    unpack8<kF16>(load8h<kVec>(a.dY + at, c, a.k), dy);
    unpack8<kF16>(load8h<kVec>(a.H + at, c, a.k), h);
    gain8<kF16>(load_gain<kVec>(a.w, a.w32, c, a.k), a.w32, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(dy[i] * (h[i] * rstd), w[i], s);
  }
  const float dot = row_sum<1024>(s, red) * a.inv_k;
  for (int64_t c = 8 * threadIdx.x; c < a.k; c += 8192) {
    float w[8];
    gain8<kF16>(load_gain<kVec>(a.w, a.w32, c, a.k), a.w32, w);
    const u32x4 r = a.R != nullptr ? load8h<kVec>(a.R + at, c, a.k) : u32x4{0u, 0u, 0u, 0u};
    store8h<kVec>(a.dX + at, c, a.k,
                  dx8<kF16>(load8h<kVec>(a.dY + at, c, a.k), load8h<kVec>(a.H + at, c, a.k), r, a.R != nullptr, rstd, dot, w));
  }
}

// dw's partial sums for rows of any length: a column per lane, a range of rows
// per workgroup row.
template <bool kF16>
__global__ __launch_bounds__(256) void rms_dw_long_kernel(BwdArgs a, int64_t rows) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m0 = blockIdx.y * rows, m1 = m0 + rows < a.M ? m0 + rows : a.M;
  if (c >= a.k) return;
  float s = 0.0f;
  for (int64_t m = m0; m < m1; ++m)
    s = fmaf(from16<kF16>(a.dY[m * a.k + c]), from16<kF16>(a.H[m * a.k + c]) * a.rstd[m], s);
  a.part[blockIdx.y * a.k + c] = s;
}

// dw (+)= the partial sums [parts][k], added in order: 64 columns per workgroup,
// 16 ranges of the parts at a time.
__global__ __launch_bounds__(1024) void rms_dw_kernel(const float* __restrict__ part, int parts, int64_t k,
                                                      float* __restrict__ dw, int accumulate) {
  __shared__ float join[16][64];
  const int lane = threadIdx.x & 63, range = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const int each = (parts + 15) / 16, p1 = (range + 1) * each < parts ? (range + 1) * each : parts;
  float s = 0.0f;
  if (c < k) {
#pragma unroll 8
    for (int p = range * each; p < p1; ++p) s += part[(int64_t)p * k + c];
  }
  join[range][lane] = s;
  __syncthreads();
  if (range != 0 || c >= k) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += join[i][lane];
  dw[c] = accumulate ? dw[c] + s : s;
}

template <bool kF16, bool kVec>
void fwd_of(const FwdArgs& a, hipStream_t st) {
#define QLORA_RMS(LPR, V) \
  rms_fwd_kernel<kF16, LPR, V, kVec><<<(unsigned)cdiv(a.M, (int64_t)(LPR < 256 ? 256 / LPR : 1)), LPR < 256 ? 256 : LPR, 0, st>>>(a)
  if (a.k > kInRegisters) rms_fwd_long_kernel<kF16, kVec><<<(unsigned)a.M, 1024, 0, st>>>(a);
  else if (a.k <= 128) QLORA_RMS(16, 1);
  else if (a.k <= 512) QLORA_RMS(64, 1);
  else if (a.k <= 1024) QLORA_RMS(64, 2);
  else if (a.k <= 2048) QLORA_RMS(256, 1);
  else if (a.k <= 4096) QLORA_RMS(256, 2);
  else if (a.k <= 8192) QLORA_RMS(256, 4);
  else if (a.k <= 16384) QLORA_RMS(512, 4);
  else QLORA_RMS(1024, 4);
#undef QLORA_RMS
}

// Workgroups of the backward with dw, and their threads: what a compute unit holds
constexpr int kDwGroups = 256, kDwThreads = 1024;

int dw_rows(int64_t k) {
  return kDwThreads / (k <= 128 ? 16 : k <= 1024 ? 64 : k <= 2048 ? 256 : k <= 8192 ? 512 : 1024);
}

int dw_parts(int64_t M, int64_t k) {
  const int64_t most = k > kInRegisters ? 64 : kDwGroups, need = k > kInRegisters ? M : cdiv(M, (int64_t)dw_rows(k));
  return (int)(need < most ? need : most);
}

template <bool kF16, bool kVec>
void bwd_of(const BwdArgs& a, hipStream_t st) {
#define QLORA_RMS(LPR, V)                                                              \
  {                                                                                    \
    constexpr int kT = LPR < 256 ? 256 : LPR;                                          \
    rms_bwd_kernel<kF16, LPR, V, kT, kVec, false>                                      \
        <<<(unsigned)cdiv(a.M, (int64_t)(kT / LPR)), kT, 0, st>>>(a);                  \
  }
#define QLORA_RMS_DW(LPR, V) \
  rms_bwd_kernel<kF16, LPR, V, kDwThreads, kVec, true><<<(unsigned)dw_parts(a.M, a.k), kDwThreads, 0, st>>>(a)
  if (a.k > kInRegisters) {
    if (a.dX != nullptr) rms_bwd_long_kernel<kF16, kVec><<<(unsigned)a.M, 1024, 0, st>>>(a);
    if (a.part != nullptr) {
      const int64_t parts = dw_parts(a.M, a.k);
      const dim3 grid((unsigned)cdiv(a.k, (int64_t)256), (unsigned)parts);
      rms_dw_long_kernel<kF16><<<grid, 256, 0, st>>>(a, cdiv(a.M, parts));
    }
  } else if (a.part == nullptr) {
    if (a.k <= 128) QLORA_RMS(16, 1)
    else if (a.k <= 512) QLORA_RMS(64, 1)
    else if (a.k <= 1024) QLORA_RMS(64, 2)
    else if (a.k <= 2048) QLORA_RMS(256, 1)
    else if (a.k <= 4096) QLORA_RMS(256, 2)
    else if (a.k <= 8192) QLORA_RMS(256, 4)
    else if (a.k <= 16384) QLORA_RMS(512, 4)
    else QLORA_RMS(1024, 4)
  } else {
    if (a.k <= 128) QLORA_RMS_DW(16, 1);
    else if (a.k <= 512) QLORA_RMS_DW(64, 1);
    else if (a.k <= 1024) QLORA_RMS_DW(64, 2);
    else if (a.k <= 2048) QLORA_RMS_DW(256, 1);
    else if (a.k <= 4096) QLORA_RMS_DW(512, 1);
    else if (a.k <= 8192) QLORA_RMS_DW(512, 2);
    else if (a.k <= 16384) QLORA_RMS_DW(1024, 2);
    else QLORA_RMS_DW(1024, 4);
  }
#undef QLORA_RMS
#undef QLORA_RMS_DW
}

}  // namespace

hipError_t launch_rms_fwd(const uint16_t* X, const uint16_t* R, const void* w, bool w32, int64_t M, int64_t k, float eps,
                          uint16_t* Y, uint16_t* H, float* rstd, uint8_t* codes, uint8_t* scale, hipStream_t st, bool f16) {
  if (codes != nullptr && k % 64 != 0) return hipErrorInvalidValue;
  const FwdArgs a = {X, R, w, w32, M, k, codes != nullptr ? f8_pad(k) : k, 1.0f / (float)k, eps, Y, H, rstd, codes, scale};
  const bool vec = k % 8 == 0;
  if (f16) vec ? fwd_of<true, true>(a, st) : fwd_of<true, false>(a, st);
  else vec ? fwd_of<false, true>(a, st) : fwd_of<false, false>(a, st);
  return hipGetLastError();
}

size_t rms_bwd_ws_bytes(int64_t M, int64_t k) { return (size_t)dw_parts(M, k) * (size_t)k * 4; }

hipError_t launch_rms_bwd(const uint16_t* dY, const uint16_t* H, const float* rstd, const void* w, bool w32,
                          const uint16_t* R, int64_t M, int64_t k, uint16_t* dX, float* dw, int accumulate, float* part,
                          hipStream_t st, bool f16) {
  const BwdArgs a = {dY, H, R, rstd, w, w32, M, k, 1.0f / (float)k, dX, dw != nullptr ? part : nullptr};
  const bool vec = k % 8 == 0;
  if (f16) vec ? bwd_of<true, true>(a, st) : bwd_of<true, false>(a, st);
  else vec ? bwd_of<false, true>(a, st) : bwd_of<false, false>(a, st);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && dw != nullptr) {
    rms_dw_kernel<<<(unsigned)cdiv(k, (int64_t)64), 1024, 0, st>>>(part, dw_parts(M, k), k, dw, accumulate);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace qlora
