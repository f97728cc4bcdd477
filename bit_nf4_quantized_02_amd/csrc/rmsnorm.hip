// Residual addition with the root-mean-square norm, and its backward.
//
//   h = RN16(RN32(x + res)),  rstd = (mean(h^2) + eps)^-1/2,  y = RN16(h rstd w)
//   g = dy w,  hn = h rstd,  dx = RN16(rstd (g - hn mean(g hn)) + dres),  dw = sum over rows of dy hn
//
// Sums are fp32; the forward joins a row's waves and takes the root in fp64, so
// that rstd is off by little more than its own rounding (4096 columns: 3.1e-8 rms, of
// which the rounding is 2.8e-8; all in fp32 4.5e-8, in the same time). The stream h is
// rounded before it is normalised: the backward, which reads it again, then
// differentiates what was computed. As 8-bit activations (fp8.h) the 16-bit y is
// encoded, so that the layer gets the same codes from here as it makes of y itself.
//
// Bound by HBM: every value is read once and stays in registers between the sum
// and its use. kLpr lanes hold a row, kV runs of 8 values each; 16 neighbouring
// lanes hold 128 columns, a scale block of the 8-bit form. Rows of more than 32768
// columns do not fit a workgroup's registers and are read twice.
//
// Measured (bf16, whole calls, three sets of operands in turn; 16 sets take the same,
// one, partly in the last-level cache, 40 us): 4096 x 8192, 268 MB, forward with
// residual 48 us (5.6 TB/s; a copy of 1 GB runs at 5.1), dX 46, with dw 54; 8-bit output
// instead of y 45 us (5.2 TB/s); 262144 x 128 50, 49 and 54; 838 x 40000 (rows read
// twice) 66, 69 and 108. One row of 8192 columns: 3 us in the kernel, 11 for a call.
#include "fp8.h"
#include "kernels.h"

namespace qlora {

namespace {

constexpr int64_t kInRegisters = 32768;  // columns of a row that a workgroup holds

// Columns that the lanes of a row have to hold: rows of no multiple of 8 are cut
// up to 7 columns before they begin.
int64_t held(int64_t k) { return k % 8 == 0 ? k : k + 7; }

// A workgroup for each of `groups`, over two dimensions where one would have 2^32
// threads or more (2^22 rows of 16378 to 16383 columns); there may be more workgroups
// than groups then. group_of(): a workgroup's place.
dim3 grid_of(int64_t groups, int threads) {
  const int64_t y = cdiv(groups * threads, (int64_t)1 << 31);
  return dim3((unsigned)cdiv(groups, y), (unsigned)y);
}
__device__ __forceinline__ int64_t group_of() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Workgroups of the backward with dw, at most: one of 1024 threads for each
// compute unit (8 M values in rows of 128 to 1024: 15 - 16 us; 512 of 512 threads 16 -
// 17, 1024 of 256 18 - 19, with more partial sums to write and read).
constexpr int kDwGroups = 256;

// Eight 16-bit values into (row, c) of any alignment, nothing from n on.
__device__ __forceinline__ void store8h(uint16_t* __restrict__ row, int64_t c, int64_t n, const u32x4& v) {
  if (c + 8 <= n) {
    *reinterpret_cast<u32x4_any*>(row + c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
  }
}

// Elements d .. of eight, zeros after them (d >= 1).
__device__ __forceinline__ void take_from(u32x4& x, int d) {
  if (d >= 8) x = u32x4{0u, 0u, 0u, 0u};
  if (d & 4) x = u32x4{x[2], x[3], 0u, 0u};
  if (d & 2) x = u32x4{x[1], x[2], x[3], 0u};
  if (d & 1)
    x = u32x4{(x[0] >> 16) | (x[1] << 16), (x[1] >> 16) | (x[2] << 16), (x[2] >> 16) | (x[3] << 16), x[3] >> 16};
}

// Zeros, then the first 8 - d elements of eight (1 <= d <= 7).
__device__ __forceinline__ void put_from(u32x4& x, int d) {
  if (d & 4) x = u32x4{0u, 0u, x[0], x[1]};
  if (d & 2) x = u32x4{0u, x[0], x[1], x[2]};
  if (d & 1)
    x = u32x4{x[0] << 16, (x[0] >> 16) | (x[1] << 16), (x[1] >> 16) | (x[2] << 16), (x[2] >> 16) | (x[3] << 16)};
}

// Elements [lo, hi) of eight to p + lo .., where lo = 0 or hi = 8: a power of two of
// them at a time. W4, W2: 8 and 4 bytes, as aligned as p is.
template <typename W4, typename W2>
__device__ __forceinline__ void store_some(uint16_t* p, const u32x4& x, int lo, int hi) {
  if (lo == 0) {
    if (hi & 4) *reinterpret_cast<W4*>(p) = u32x2{x[0], x[1]};
    if (hi & 2) *reinterpret_cast<W2*>(p + (hi & 4)) = hi & 4 ? x[2] : x[0];
    if (hi & 1) p[hi - 1] = (uint16_t)(hi & 4 ? (hi & 2 ? x[3] : x[2]) : (hi & 2 ? x[1] : x[0]));
  } else {
    const int n = 8 - lo;
    if (n & 1) p[lo] = (uint16_t)((n & 4 ? (n & 2 ? x[0] : x[1]) : (n & 2 ? x[2] : x[3])) >> 16);
    if (n & 2) *reinterpret_cast<W2*>(p + (n & 4 ? 2 : 6)) = n & 4 ? x[1] : x[3];
    if (n & 4) *reinterpret_cast<W4*>(p + 4) = u32x2{x[2], x[3]};
  }
}

// A wave's first row and, where it has several, the lane's place among them.
struct Place {
  int64_t first;  // (the same in all lanes)
  int lead;
  __device__ __forceinline__ int64_t row() const { return first + lead; }
  __device__ __forceinline__ Place after(int64_t rows) const { return Place{first + rows, lead}; }
};

// The thread's place in a workgroup whose first row is m0.
template <int kLpr>
__device__ __forceinline__ Place place_of(int64_t m0) {
  static_assert(kLpr == 16 || kLpr == 32 || kLpr >= 64, "a wave has four rows, two or one");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if constexpr (kLpr >= 64) return Place{m0 + wave / (kLpr / 64), 0};
  else return Place{m0 + 64 / kLpr * wave, (int)(threadIdx.x & 63) / kLpr};
}

// A row of [M, k] 16-bit values, read and written in runs of eight by the kLpr
// lanes that hold it: run v of lane t begins at column 8 (t + kLpr v) - shift.
//
// Rows go through buffer descriptors, whose range check replaces a branch at each
// run (a load behind one waits for the one before it) and whose addresses take few
// vector registers: a descriptor of the row where a wave has one only, else of
// the wave's rows. A row past the last reads as zeros. Rows whose length is no
// multiple of 8 (kVec false) start anywhere: their runs are cut at multiples of 16
// bytes all the same, from `shift` columns before the row, so that loads and stores
// are aligned (5001 columns: unaligned runs 72 us for 268 MB, aligned 55). finish()
// clears what a run holds of the row before; the last column of an odd end, of
// whose word half is out of range, is loaded apart (tail()).
// Several short rows in a wave with such lengths are read and written by address:
// a run that reaches past its row is read from the row's last eight values, which
// finish() moves into place (a branch with loads of its own waits for those before
// it: 71 columns 124 us for 268 MB).
template <int kLpr, bool kVec>
struct RowOf {
  static constexpr bool kShift = !kVec && kLpr >= 64, kAddress = !kVec && kLpr < 64;
  i32x4 rs;
  int off, shift, end;  // end: of the row, counted as the runs' columns + shift
  uint16_t* p;
  __device__ __forceinline__ RowOf(const uint16_t* base, const Place& at, int64_t M, int64_t k, int t) {
    uint16_t* const b = const_cast<uint16_t*>(base);
    shift = 0;
    if constexpr (kAddress) {
      p = b + (at.row() < M ? at.row() : M - 1) * k;
    } else if constexpr (kLpr >= 64) {
      p = b + at.first * k;
      if constexpr (kShift) shift = shift_of(at, k);
      rs = make_rsrc(p - shift, at.first < M ? 2 * (k + shift) : 0);
      off = 16 * t;
    } else {
      const int64_t left = M - at.first;
      rs = make_rsrc(b + at.first * k, left > 0 ? 2 * k * (left < 64 / kLpr ? left : 64 / kLpr) : 0);
      off = 8 * t < k ? 2 * (int)k * at.lead + 16 * t : -1;  // (-1: past every row)
    }
    end = (int)k + shift;
  }
  static __device__ __forceinline__ int shift_of(const Place& at, int64_t k) {
    return kShift ? (int)((at.first * k) & 7) : 0;
  }
  __device__ __forceinline__ u32x4 load(int t, int v) const {
    const int c = 8 * (t + kLpr * v);
    if constexpr (kAddress)
      return end < 8 ? load8h<false>(p, c, end) : *reinterpret_cast<const u32x4_any*>(p + (c + 8 <= end ? c : end - 8));
    else return raw_buffer_load_b128(rs, off, 16 * kLpr * v, 0);
  }
  __device__ __forceinline__ uint32_t tail() const {
    if constexpr (kShift) return end & 1 ? raw_buffer_load_u16(rs, 2 * end - 2, 0, 0) : 0u;
    else return 0u;
  }
  static __device__ __forceinline__ void finish(u32x4& x, uint32_t tail, int shift, int64_t k, int t, int v) {
    if constexpr (kShift) {
      const int e = 8 * (t + kLpr * v), last = (int)k + shift - 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (v == 0) {
          if (e + 2 * i < shift) x[i] &= 0xFFFF0000u;
          if (e + 2 * i + 1 < shift) x[i] = 0u;
        }
        if (!(last & 1) && e + 2 * i == last) x[i] = tail;
      }
    }
    if constexpr (kAddress) {
      const int past = 8 * (t + kLpr * v) + 8 - (int)k;
      if (k >= 8 && past > 0) take_from(x, past);
    }
  }
  __device__ __forceinline__ void store(int t, int v, const u32x4& x) const {
    if constexpr (kAddress) {
      typedef u32x2 __attribute__((aligned(2))) W4;
      typedef uint32_t __attribute__((aligned(2))) W2;
      const int c = 8 * (t + kLpr * v);
      if (c + 8 <= end) *reinterpret_cast<u32x4_any*>(p + c) = x;
      else if (c < end) store_some<W4, W2>(p + c, x, 0, end - c);
    } else if constexpr (!kShift) {
      buffer_store16(rs, off + 16 * kLpr * v, x);
    } else {
      const int e = 8 * (t + kLpr * v);
      const bool whole = e >= shift && e + 8 <= end;
      buffer_store16(rs, whole ? off + 16 * kLpr * v : -1, x);
      if (!whole && e < end)
        store_some<u32x2, uint32_t>(p + (e - shift), x, e < shift ? shift - e : 0, end - e < 8 ? end - e : 8);
    }
  }
};

// Eight gains from c on, as they are stored: in 16 bits or (kW32) fp32.
template <bool kW32>
struct Gain {
  u32x4 a[kW32 ? 2 : 1];
};

// A run that reaches past w's ends is read from its first or last eight gains;
// settle() moves them into place and clears the others, apart from the loads, so
// that nothing waits between these (an edge that loads its gains one by one, behind
// a branch: 4103 columns 66 us for 268 MB).
template <bool kW32, bool kVec>
__device__ __forceinline__ Gain<kW32> load_gain(const void* __restrict__ w, int64_t c, int64_t n) {
  Gain<kW32> g;
#pragma unroll
  for (int i = 0; i < (kW32 ? 2 : 1); ++i) g.a[i] = u32x4{0u, 0u, 0u, 0u};
  if (kVec ? c >= n : n < 8) {
    if constexpr (!kVec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c + i < 0 || c + i >= n) continue;
        if constexpr (kW32) g.a[i >> 2][i & 3] = static_cast<const uint32_t*>(w)[c + i];
        else g.a[0][i >> 1] |= (uint32_t)static_cast<const uint16_t*>(w)[c + i] << (16 * (i & 1));
      }
    }
    return g;
  }
  if constexpr (!kVec) c = c < 0 ? 0 : c + 8 <= n ? c : n - 8;
  if constexpr (kW32) {
    typedef u32x4 __attribute__((aligned(4))) u32x4_4;
    const uint32_t* const p = static_cast<const uint32_t*>(w) + c;
    g.a[0] = *reinterpret_cast<const u32x4_4*>(p);
    g.a[1] = *reinterpret_cast<const u32x4_4*>(p + 4);
  } else if constexpr (kVec) {
    g.a[0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(w) + c);
  } else {
    g.a[0] = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(w) + c);
  }
  return g;
}

template <bool kW32, bool kVec>
__device__ __forceinline__ void settle(Gain<kW32>& g, int64_t c, int64_t n) {
  if (kVec || n < 8) return;
  const int past = c + 8 <= n ? 0 : c + 8 - n < 8 ? (int)(c + 8 - n) : 8, before = c < 0 ? (int)-c : 0;
  if constexpr (!kW32) {
    if (past > 0) take_from(g.a[0], past);
    if (before > 0) put_from(g.a[0], before);
  } else if (past > 0 || before > 0) {
    uint32_t f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = past < 8 ? g.a[i >> 2][i & 3] : 0u;
#pragma unroll
    for (int b = 4; b > 0; b /= 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = past & b ? (i + b < 8 ? f[i + b < 8 ? i + b : 0] : 0u) : f[i];
#pragma unroll
      for (int i = 7; i >= 0; --i) f[i] = before & b ? (i >= b ? f[i >= b ? i - b : 0] : 0u) : f[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) g.a[i >> 2][i & 3] = f[i];
  }
}

template <bool kF16, bool kW32>
__device__ __forceinline__ void gain8(const Gain<kW32>& g, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (kW32) f[i] = __uint_as_float(g.a[i >> 2][i & 3]);
    else f[i] = from16<kF16>((g.a[0][i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
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
template <int kCtrl>
__device__ __forceinline__ double rotated(double x) {
  return __hiloint2double(__builtin_amdgcn_mov_dpp(__double2hiint(x), kCtrl, 0xF, 0xF, true),
                          __builtin_amdgcn_mov_dpp(__double2loint(x), kCtrl, 0xF, 0xF, true));
}

// Sum over the kLpr lanes of a row, in all of them and in one order always; the
// sums of several waves are added as F. In fp64 each of 16 lanes takes one and they
// are added in pairs (all 16 in every lane: 55.8 us against 54.6 at 22016 columns).
// red: one float for each wave of the workgroup, used when a row has more than
// one wave (then every thread of the workgroup calls).
template <int kLpr, typename F = float>
__device__ __forceinline__ F row_sum(float s, float* red) {
  s += rotated<0x128>(s);
  s += rotated<0x124>(s);
  s += rotated<0x122>(s);
  s += rotated<0x121>(s);
  if constexpr (kLpr >= 32) s += __shfl_xor(s, 16);
  if constexpr (kLpr >= 64) s += __shfl_xor(s, 32);
  if constexpr (kLpr > 64) {
    constexpr int kWaves = kLpr / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = s;
    __syncthreads();
    if constexpr (sizeof(F) == sizeof(float)) {
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) s += red[wave / kWaves * kWaves + i];
    } else {
      F p = (F)red[wave / kWaves * kWaves + (threadIdx.x & (kWaves - 1))];
      if constexpr (kWaves == 16) p += rotated<0x128>(p);
      if constexpr (kWaves >= 8) p += rotated<0x124>(p);
      if constexpr (kWaves >= 4) p += rotated<0x122>(p);
      p += rotated<0x121>(p);
      return p;
    }
  }
  return (F)s;
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

// Sum of the squares of eight values (each exact in fp32), in pairs.
template <bool kF16>
__device__ __forceinline__ float squares8(const u32x4& h) {
  float f[8];
  unpack8<kF16>(h, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = fmaf(f[i], f[i], f[i + 4] * f[i + 4]);
  return (f[0] + f[2]) + (f[1] + f[3]);
}

// x^-1/2 to within a rounding: the instruction's value (1 ulp) and one step of
// Newton's method in fp64. Outside the range where that holds, 0 and infinity
// among it, in fp32.
__device__ __forceinline__ float rstd_of(double x) {
  if (x > 1e-37 && x < 1e38) {
    const double d = (double)__builtin_amdgcn_rsqf((float)x);
    return (float)(d * fma(-0.5 * x * d, d, 1.5));
  }
  return 1.0f / sqrtf((float)x);
}

// y of eight values, in 16 bits. With w of 16 bits h w is exact in fp32, and the
// product with rstd is the only rounding before y's own. In bf16 the power of two in
// rstd goes to h first (exact as well, down to 2^-126): |h w| alone may be anything
// from 2^-266 to 2^256 where h rstd w is an ordinary number. A rstd of 0, infinity or
// NaN stays what it is in the products. (Times as without the power, within 1%.)
template <bool kF16, bool kW32>
__device__ __forceinline__ u32x4 normed8(const u32x4& h, float rstd, const Gain<kW32>& g) {
  float f[8], w[8];
  unpack8<kF16>(h, f);
  gain8<kF16>(g, w);
  const uint32_t b = __float_as_uint(rstd);
  const float power = __uint_as_float(b & 0x7F800000u);
  const float rest = isnan(rstd) ? rstd : __uint_as_float((b & 0x7FFFFFu) | 0x3F800000u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (kW32) f[i] = f[i] * rstd * w[i];
    else if constexpr (kF16) f[i] = f[i] * w[i] * rstd;
    else f[i] = f[i] * power * w[i] * rest;
  }
  return pack8<kF16>(f);
}

// The 8-bit form of y: 16 neighbouring lanes (all of them call) hold a block of
// 128 columns and find its scale; columns c .. of row m are this lane's. Those
// from k on are zero, whatever the row's rstd has made of them.
template <bool kF16>
__device__ __forceinline__ void encode8(u32x4 y, int64_t m, int64_t c, int64_t k, int64_t kp, uint8_t* __restrict__ codes,
                                        uint8_t* __restrict__ scale) {
  if (c >= k) y = u32x4{0u, 0u, 0u, 0u};
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
  int64_t M, k, kp;
  double inv_k;
  float eps;
  uint16_t *Y, *H;        // Y may be NULL; H is there if R is
  float* rstd;            // may be NULL
  uint8_t *codes, *scale; // may be NULL
};

// 1024 threads with a 16-bit gain take at most 64 registers each, for two workgroups
// on a compute unit: bf16 64 instead of 66 (four values a lane in scratch: 28672
// columns to 8 bits 50 us against 53, 22016 50 and 54; 256 and 512 threads lose 2 us of
// 47 by it), fp16 62 either way. Gains of 32 bits, 82 and 75 registers, would put 39 and
// 26 into scratch (28672 columns to 16 bits: bf16 92 us against 54, fp16 74 against 54).
template <bool kF16, bool kW32, int kLpr, int kV, bool kVec>
__global__ __attribute__((amdgpu_waves_per_eu(kLpr == 1024 && kVec && !kW32 ? 8 : 1))) __launch_bounds__(
    kLpr < 256 ? 256 : kLpr) void rms_fwd_kernel(FwdArgs a) {
  constexpr int kThreads = kLpr < 256 ? 256 : kLpr;
  __shared__ float red[kThreads / 64];
  const int t = threadIdx.x & (kLpr - 1);
  const Place at = place_of<kLpr>(group_of() * (kThreads / kLpr));
  const int64_t m = at.row();
  const bool live = m < a.M;
  typedef RowOf<kLpr, kVec> Row;
  const Row X(a.X, at, a.M, a.k, t);
  u32x4 h[kV], r[kV];
  uint32_t xt = X.tail(), rt = 0;
  Gain<kW32> g[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) h[v] = X.load(t, v);
  if (a.R != nullptr) {
    const Row R(a.R, at, a.M, a.k, t);
    rt = R.tail();
#pragma unroll
    for (int v = 0; v < kV; ++v) r[v] = R.load(t, v);
  }
#pragma unroll
  for (int v = 0; v < kV; ++v) g[v] = load_gain<kW32, kVec>(a.w, 8 * (t + kLpr * v) - X.shift, a.k);
#pragma unroll
  for (int v = 0; v < kV; ++v) Row::finish(h[v], xt, X.shift, a.k, t, v);
  if (a.R != nullptr) {
    const Row H(a.H, at, a.M, a.k, t);
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      Row::finish(r[v], rt, X.shift, a.k, t, v);
      h[v] = add8<kF16>(h[v], r[v]);
      if (live) H.store(t, v, h[v]);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < kV; ++v) s += squares8<kF16>(h[v]);
  const float rstd = rstd_of(fma(row_sum<kLpr, double>(s, red), a.inv_k, (double)a.eps));
  if (!live) return;
  if (t == 0 && a.rstd != nullptr) a.rstd[m] = rstd;
  const Row Y(a.Y, at, a.M, a.k, t);
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int64_t c = 8 * (t + kLpr * v);
    settle<kW32, kVec>(g[v], c - X.shift, a.k);
    const u32x4 y = normed8<kF16>(h[v], rstd, g[v]);
    if (a.Y != nullptr) Y.store(t, v, y);
    if (kVec && a.codes != nullptr && c < a.kp) encode8<kF16>(y, m, c, a.k, a.kp, a.codes, a.scale);
  }
}

// Rows of any length, read twice (the second time from the caches, if they hold
// a row of every workgroup).
template <bool kF16, bool kW32, bool kVec>
__global__ __launch_bounds__(1024) void rms_fwd_long_kernel(FwdArgs a) {
  __shared__ float red[16];
  const int64_t m = blockIdx.x, at = m * a.k;
  const uint16_t* const in = a.R != nullptr ? a.H + at : a.X + at;
  float s = 0.0f;
  for (int64_t c = 8 * threadIdx.x; c < a.k; c += 8192) {
    u32x4 h = load8h<kVec>(a.X + at, c, a.k);
    if (a.R != nullptr) {
      h = add8<kF16>(h, load8h<kVec>(a.R + at, c, a.k));
      store8h(a.H + at, c, a.k, h);
    }
    s += squares8<kF16>(h);
  }
  const float rstd = rstd_of(fma(row_sum<1024, double>(s, red), a.inv_k, (double)a.eps));
  if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[m] = rstd;
  for (int64_t c = 8 * threadIdx.x; c < a.kp; c += 8192) {  // (each thread reads what it wrote)
    Gain<kW32> g = load_gain<kW32, kVec>(a.w, c, a.k);
    settle<kW32, kVec>(g, c, a.k);
    const u32x4 y = normed8<kF16>(load8h<kVec>(in, c, a.k), rstd, g);
    if (a.Y != nullptr) store8h(a.Y + at, c, a.k, y);
    if (kVec && a.codes != nullptr) encode8<kF16>(y, m, c, a.k, a.kp, a.codes, a.scale);
  }
}

struct BwdArgs {
  const uint16_t *dY, *H, *R;  // R: the gradient that reaches h past the norm, or NULL
  const float* rstd;
  const void* w;
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

// One row's share of a lane, as it was loaded.
template <int kV>
struct RowRegs {
  u32x4 dy[kV], h[kV], r[kV];
  uint32_t tail[3];
  float rstd;
};

template <int kLpr, int kV, bool kVec>
__device__ __forceinline__ void load_row(const BwdArgs& a, const Place& at, int t, RowRegs<kV>& x) {
  const RowOf<kLpr, kVec> dY(a.dY, at, a.M, a.k, t), H(a.H, at, a.M, a.k, t);
  x.tail[0] = dY.tail();
  x.tail[1] = H.tail();
  x.tail[2] = 0;
#pragma unroll
  for (int v = 0; v < kV; ++v) x.dy[v] = dY.load(t, v);
#pragma unroll
  for (int v = 0; v < kV; ++v) x.h[v] = H.load(t, v);
  if (!RowOf<kLpr, kVec>::kAddress || a.R != nullptr) {
    const RowOf<kLpr, kVec> R(a.R, at, a.R != nullptr ? a.M : 0, a.k, t);  // (no R: rows past the last)
    x.tail[2] = R.tail();
#pragma unroll
    for (int v = 0; v < kV; ++v) x.r[v] = R.load(t, v);
  } else {
#pragma unroll
    for (int v = 0; v < kV; ++v) x.r[v] = u32x4{0u, 0u, 0u, 0u};
  }
  x.rstd = a.rstd[at.row() < a.M ? at.row() : a.M - 1];
}

// Where a lane's sums of dw are: nowhere, in registers, or in LDS (f32x4 of the
// lane's half-run h of run v at (2 v + h) kLpr + t).
enum class Dw { kNone, kRegs, kLds };

// A row's dx from its registers, and dy hn added to the sums of dw. Every thread
// of the workgroup calls (row_sum).
template <bool kF16, bool kW32, int kLpr, int kV, bool kVec, Dw kDw>
__device__ __forceinline__ void do_row(const BwdArgs& a, const Place& at, int t, RowRegs<kV>& x, const Gain<kW32> (&g)[kV],
                                       float (&acc)[kDw == Dw::kRegs ? kV : 1][8], f32x4* lds, float* red) {
  const bool live = at.row() < a.M;
  const int shift = RowOf<kLpr, kVec>::shift_of(at, a.k);
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    RowOf<kLpr, kVec>::finish(x.dy[v], x.tail[0], shift, a.k, t, v);
    RowOf<kLpr, kVec>::finish(x.h[v], x.tail[1], shift, a.k, t, v);
    RowOf<kLpr, kVec>::finish(x.r[v], x.tail[2], shift, a.k, t, v);
    float dy[8], h[8], w[8];
    unpack8<kF16>(x.dy[v], dy);
    unpack8<kF16>(x.h[v], h);
    gain8<kF16>(g[v], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = dy[i] * (h[i] * x.rstd);
      s = fmaf(p, w[i], s);
      if constexpr (kDw == Dw::kRegs) acc[v][i] += live ? p : 0.0f;
      dy[i] = p;
    }
    if constexpr (kDw == Dw::kLds) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        lds[(2 * v + j) * kLpr + t] += f32x4{dy[4 * j], dy[4 * j + 1], dy[4 * j + 2], dy[4 * j + 3]};
    }
  }
  const float dot = row_sum<kLpr>(s, red) * a.inv_k;
  if (!live || a.dX == nullptr) return;
  const RowOf<kLpr, kVec> dX(a.dX, at, a.M, a.k, t);
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    // (unpacked again: kept from above, the fp32 values take twice the registers)
    asm volatile("" : "+v"(x.dy[v]), "+v"(x.h[v]));
    float w[8];
    gain8<kF16>(g[v], w);
    dX.store(t, v, dx8<kF16>(x.dy[v], x.h[v], x.r[v], a.R != nullptr, x.rstd, dot, w));
  }
}

// dX alone: a row for each kLpr threads.
template <bool kF16, bool kW32, int kLpr, int kV, bool kVec>
__global__ __launch_bounds__(kLpr < 256 ? 256 : kLpr) void rms_dx_kernel(BwdArgs a) {
  constexpr int kThreads = kLpr < 256 ? 256 : kLpr;
  __shared__ float red[kThreads / 64];
  const int t = threadIdx.x & (kLpr - 1);
  const Place at = place_of<kLpr>(group_of() * (kThreads / kLpr));
  RowRegs<kV> x;
  Gain<kW32> g[kV];
  float none[1][8];
  load_row<kLpr, kV, kVec>(a, at, t, x);
#pragma unroll
  for (int v = 0; v < kV; ++v)
    g[v] = load_gain<kW32, kVec>(a.w, 8 * (t + kLpr * v) - RowOf<kLpr, kVec>::shift_of(at, a.k), a.k);
#pragma unroll
  for (int v = 0; v < kV; ++v)
    settle<kW32, kVec>(g[v], 8 * (t + kLpr * v) - RowOf<kLpr, kVec>::shift_of(at, a.k), a.k);
  do_row<kF16, kW32, kLpr, kV, kVec, Dw::kNone>(a, at, t, x, g, none, nullptr, red);
}

// dX and dw: kThreads threads hold kThreads / kLpr rows at a time and walk over the
// rows with the grid, the next rows loaded before this one's sum. Each lane adds up dy
// hn of its columns over the rows it meets; the rows of a workgroup are joined in LDS
// at the end, the workgroups by rms_dw_kernel.
template <bool kF16, bool kW32, int kLpr, int kV, int kThreads, bool kVec>
__global__ __launch_bounds__(kThreads) void rms_bwd_kernel(BwdArgs a) {
  constexpr int kRows = kThreads / kLpr, kCols = 8 * kLpr * kV;
  __shared__ float red[2][kThreads / 64];  // in turn: one barrier a row
  const int t = threadIdx.x & (kLpr - 1);
  const int64_t m0 = (int64_t)blockIdx.x * kRows;
  Place at = place_of<kLpr>(m0);
  // (the same for all rows of a lane: where it has more than one, they are a
  // multiple of 8 apart)
  const int shift = RowOf<kLpr, kVec>::shift_of(at, a.k);
  Gain<kW32> g[kV];
  float acc[kV][8];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    g[v] = load_gain<kW32, kVec>(a.w, 8 * (t + kLpr * v) - shift, a.k);
    settle<kW32, kVec>(g[v], 8 * (t + kLpr * v) - shift, a.k);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * kRows;
  const auto load = [&](const Place& at, RowRegs<kV>& x) { load_row<kLpr, kV, kVec>(a, at, t, x); };
  const auto row = [&](const Place& at, RowRegs<kV>& x, int turn) {
    do_row<kF16, kW32, kLpr, kV, kVec, Dw::kRegs>(a, at, t, x, g, acc, nullptr, red[turn]);
  };
  RowRegs<kV> x0, x1;
  load(at, x0);
  for (int64_t left = (a.M - m0 + step - 1) / step; left > 0; left -= 2) {
    load(at.after(step), x1);
    row(at, x0, 0);
    if (left == 1) break;
    at = at.after(step);
    load(at.after(step), x0);
    row(at, x1, 1);
    at = at.after(step);
  }
  float* const out = a.part + (int64_t)blockIdx.x * a.k;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = 8 * (t + kLpr * v) + i - shift;
        if (c >= 0 && c < a.k) out[c] = acc[v][i];
      }
  } else {
    __shared__ float join[kRows][kCols];
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = 8 * (t + kLpr * v) + i - shift;
        if (c >= 0) join[threadIdx.x / kLpr][c] = acc[v][i];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < kCols && c < a.k; c += kThreads) {
      float s = join[0][c];
#pragma unroll 8
      for (int i = 1; i < kRows; ++i) s += join[i][c];
      out[c] = s;
    }
  }
}

// dX and dw for rows that leave no registers for the sums of dw, above 8192 columns
// or 4096 with unaligned ends: those are in LDS, 4 bytes a column, each lane's its own
// (a row of 28672 columns costs a compute unit 0.9 us there and 11 us at its share of
// HBM). One row at a time, and one workgroup on a compute unit: nothing is in flight
// while a row is summed (28672 columns, 268 MB: 67 us with 28 MB of partial sums
// written, and 6 to add them).
template <bool kF16, bool kW32, int kV, bool kVec>
__global__ __launch_bounds__(1024) void rms_bwd_wide_kernel(BwdArgs a) {
  __shared__ float red[2][16];
  __shared__ f32x4 sums[2 * 1024 * kV];
  const int t = threadIdx.x;
  const int shift = RowOf<1024, kVec>::shift_of(Place{blockIdx.x, 0}, a.k);  // (of all its rows, a multiple of 8 apart)
  Gain<kW32> g[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    g[v] = load_gain<kW32, kVec>(a.w, 8 * (t + 1024 * v) - shift, a.k);
    settle<kW32, kVec>(g[v], 8 * (t + 1024 * v) - shift, a.k);
    sums[2 * v * 1024 + t] = sums[(2 * v + 1) * 1024 + t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  float none[1][8];
  RowRegs<kV> x;
  int turn = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    load_row<1024, kV, kVec>(a, Place{m, 0}, t, x);
    do_row<kF16, kW32, 1024, kV, kVec, Dw::kLds>(a, Place{m, 0}, t, x, g, none, sums, red[turn]);
  }
  float* const out = a.part + (int64_t)blockIdx.x * a.k;
#pragma unroll
  for (int v = 0; v < kV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = 8 * (t + 1024 * v) + i - shift;
      if (c >= 0 && c < a.k) out[c] = sums[(2 * v + i / 4) * 1024 + t][i & 3];
    }
}

// dX for rows of any length, one workgroup a row, which is read twice.
template <bool kF16, bool kW32, bool kVec>
__global__ __launch_bounds__(1024) void rms_bwd_long_kernel(BwdArgs a) {
  __shared__ float red[16];
  const int64_t at = (int64_t)blockIdx.x * a.k;
  const float rstd = a.rstd[blockIdx.x];
  float s = 0.0f;
  for (int64_t c = 8 * threadIdx.x; c < a.k; c += 8192) {
    float dy[8], h[8], w[8];
    unpack8<kF16>(load8h<kVec>(a.dY + at, c, a.k), dy);
    unpack8<kF16>(load8h<kVec>(a.H + at, c, a.k), h);
    Gain<kW32> g = load_gain<kW32, kVec>(a.w, c, a.k);
    settle<kW32, kVec>(g, c, a.k);
    gain8<kF16>(g, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(dy[i] * (h[i] * rstd), w[i], s);
  }
  const float dot = row_sum<1024>(s, red) * a.inv_k;
  for (int64_t c = 8 * threadIdx.x; c < a.k; c += 8192) {
    float w[8];
    Gain<kW32> g = load_gain<kW32, kVec>(a.w, c, a.k);
    settle<kW32, kVec>(g, c, a.k);
    gain8<kF16>(g, w);
    const u32x4 r = a.R != nullptr ? load8h<kVec>(a.R + at, c, a.k) : u32x4{0u, 0u, 0u, 0u};
    store8h(a.dX + at, c, a.k,
                  dx8<kF16>(load8h<kVec>(a.dY + at, c, a.k), load8h<kVec>(a.H + at, c, a.k), r, a.R != nullptr, rstd, dot, w));
  }
}

// dw's partial sums apart from dX, for rows that do not fit a workgroup: 8 columns
// per lane, a range of rows per workgroup row.
template <bool kF16, bool kVec>
__global__ __launch_bounds__(256) void rms_dw_part_kernel(BwdArgs a, int64_t rows) {
  const int64_t c = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  const int64_t m0 = blockIdx.y * rows, m1 = m0 + rows < a.M ? m0 + rows : a.M;
  if (c >= a.k) return;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int64_t m = m0; m < m1; ++m) {
    float dy[8], h[8];
    unpack8<kF16>(load8h<kVec>(a.dY + m * a.k, c, a.k), dy);
    unpack8<kF16>(load8h<kVec>(a.H + m * a.k, c, a.k), h);
    const float r = a.rstd[m];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += dy[i] * (h[i] * r);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < a.k) a.part[blockIdx.y * a.k + c + i] = s[i];
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
#pragma unroll 16
    for (int p = range * each; p < p1; ++p) s += part[(int64_t)p * k + c];
  }
  join[range][lane] = s;
  __syncthreads();
  if (range != 0 || c >= k) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += join[i][lane];
  dw[c] = accumulate ? dw[c] + s : s;
}

// Lanes of a row and runs of a lane: a workgroup of 256 threads as far as four
// runs reach (8192 columns, forward: 47.3 us; 512 lanes of two runs 47.8, 1024 of one
// 49.1; 5120: 47.2, 48.8 and 51.5), and fewer lanes than a wave's for short rows.
template <bool kF16, bool kW32, bool kVec>
struct Forward {
  static void launch(const FwdArgs& a, hipStream_t st) {
#define QLORA_RMS(LPR, V)                                                                                        \
  rms_fwd_kernel<kF16, kW32, LPR, V, kVec>                                                                       \
      <<<grid_of(cdiv(a.M, (int64_t)(LPR < 256 ? 256 / LPR : 1)), LPR < 256 ? 256 : LPR), LPR < 256 ? 256 : LPR, 0, st>>>(a)
    const int64_t k = held(a.k);
    if (k > kInRegisters) rms_fwd_long_kernel<kF16, kW32, kVec><<<(unsigned)a.M, 1024, 0, st>>>(a);
    else if (k <= 128) QLORA_RMS(16, 1);
    else if (k <= 256) QLORA_RMS(32, 1);
    else if (k <= 512) QLORA_RMS(64, 1);
    else if (k <= 1024) QLORA_RMS(64, 2);
    else if (k <= 2048) QLORA_RMS(256, 1);
    else if (k <= 4096) QLORA_RMS(256, 2);
    else if (k <= 8192) QLORA_RMS(256, 4);
    else if (k <= 16384) QLORA_RMS(512, 4);
    else QLORA_RMS(1024, 4);
#undef QLORA_RMS
  }
};

template <bool kF16, bool kW32, bool kVec>
struct DxOnly {
  static void launch(const BwdArgs& a, hipStream_t st) {
#define QLORA_RMS(LPR, V)                                                                                        \
  rms_dx_kernel<kF16, kW32, LPR, V, kVec>                                                                        \
      <<<grid_of(cdiv(a.M, (int64_t)(LPR < 256 ? 256 / LPR : 1)), LPR < 256 ? 256 : LPR), LPR < 256 ? 256 : LPR, 0, st>>>(a)
    const int64_t k = held(a.k);
    if (k > kInRegisters) rms_bwd_long_kernel<kF16, kW32, kVec><<<(unsigned)a.M, 1024, 0, st>>>(a);
    else if (k <= 128) QLORA_RMS(16, 1);
    else if (k <= 256) QLORA_RMS(32, 1);
    else if (k <= 512) QLORA_RMS(64, 1);
    else if (k <= 1024) QLORA_RMS(64, 2);
    else if (k <= 2048) QLORA_RMS(256, 1);
    else if (k <= 4096) QLORA_RMS(256, 2);
    else if (k <= 8192) QLORA_RMS(256, 4);
    else if (k <= 16384) QLORA_RMS(512, 4);
    else QLORA_RMS(1024, 4);
#undef QLORA_RMS
  }
};

// Rows that a workgroup of the backward with dw holds at a time. Two of up to
// 8192 columns, 16 values a lane, rather than one (5120: 54 us against 59, 8192: 55
// and 56, for 268 MB); not with unaligned ends, which leave such a lane no registers:
// one, and the sums of dw in LDS (5001: 71 us; in registers 74, two rows 93).
int dw_rows(int64_t k) {
  const int64_t most2 = k % 8 == 0 ? 8192 : 4096;
  k = held(k);
  return k <= 128 ? 64 : k <= 256 ? 32 : k <= 512 ? 16 : k <= 1024 ? 8 : k <= 2048 ? 4 : k <= most2 ? 2 : 1;
}

int dw_parts(int64_t M, int64_t k) {
  const bool fits = held(k) <= kInRegisters;
  const int64_t most = fits ? kDwGroups : 128, need = fits ? cdiv(M, (int64_t)dw_rows(k)) : M;
  return (int)(need < most ? need : most);
}

template <bool kF16, bool kW32, bool kVec>
struct Backward {
  static void launch(const BwdArgs& a, hipStream_t st) {
    const int64_t parts = dw_parts(a.M, a.k), k = held(a.k);
#define QLORA_WIDE(V) rms_bwd_wide_kernel<kF16, kW32, V, kVec><<<(unsigned)parts, 1024, 0, st>>>(a)
#define QLORA_RMS(LPR, V, T) rms_bwd_kernel<kF16, kW32, LPR, V, T, kVec><<<(unsigned)parts, T, 0, st>>>(a)
    if (k > kInRegisters) {
      if (a.dX != nullptr) DxOnly<kF16, kW32, kVec>::launch(a, st);
      const dim3 grid((unsigned)cdiv(a.k, (int64_t)2048), (unsigned)parts);
      rms_dw_part_kernel<kF16, kVec><<<grid, 256, 0, st>>>(a, cdiv(a.M, parts));
    } else if (k <= 128) QLORA_RMS(16, 1, 1024);
    else if (k <= 256) QLORA_RMS(32, 1, 1024);
    else if (k <= 512) QLORA_RMS(64, 1, 1024);
    else if (k <= 1024) QLORA_RMS(128, 1, 1024);
    else if (k <= 2048) QLORA_RMS(256, 1, 1024);
    else if (k <= 4096) QLORA_RMS(512, 1, 1024);
    else if (k <= 8192) {
      if constexpr (kVec) QLORA_RMS(512, 2, 1024);
      else QLORA_WIDE(1);
    } else if (k <= 16384) QLORA_WIDE(2);
    else QLORA_WIDE(4);
#undef QLORA_RMS
#undef QLORA_WIDE
  }
};

// The variant for the types and the rows' alignment.
template <template <bool, bool, bool> class Op, typename Args>
void launch(const Args& a, bool f16, bool w32, hipStream_t st) {
  const bool vec = a.k % 8 == 0;
  if (f16) {
    if (w32) vec ? Op<true, true, true>::launch(a, st) : Op<true, true, false>::launch(a, st);
    else vec ? Op<true, false, true>::launch(a, st) : Op<true, false, false>::launch(a, st);
  } else {
    if (w32) vec ? Op<false, true, true>::launch(a, st) : Op<false, true, false>::launch(a, st);
    else vec ? Op<false, false, true>::launch(a, st) : Op<false, false, false>::launch(a, st);
  }
}

}  // namespace

hipError_t launch_rms_fwd(const uint16_t* X, const uint16_t* R, const void* w, bool w32, int64_t M, int64_t k, float eps,
                          uint16_t* Y, uint16_t* H, float* rstd, uint8_t* codes, uint8_t* scale, hipStream_t st, bool f16) {
  if (codes != nullptr && k % 64 != 0) return hipErrorInvalidValue;
  const FwdArgs a = {X, R, w, M, k, codes != nullptr ? f8_pad(k) : k, 1.0 / (double)k, eps, Y, H, rstd, codes, scale};
  launch<Forward>(a, f16, w32, st);
  return hipGetLastError();
}

size_t rms_bwd_ws_bytes(int64_t M, int64_t k) { return (size_t)dw_parts(M, k) * (size_t)k * 4; }

hipError_t launch_rms_bwd(const uint16_t* dY, const uint16_t* H, const float* rstd, const void* w, bool w32,
                          const uint16_t* R, int64_t M, int64_t k, uint16_t* dX, float* dw, int accumulate, float* part,
                          hipStream_t st, bool f16) {
  const BwdArgs a = {dY, H, R, rstd, w, M, k, 1.0f / (float)k, dX, dw != nullptr ? part : nullptr};
  if (dw != nullptr) launch<Backward>(a, f16, w32, st);
  else launch<DxOnly>(a, f16, w32, st);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && dw != nullptr) {
    rms_dw_kernel<<<(unsigned)cdiv(k, (int64_t)64), 1024, 0, st>>>(part, dw_parts(M, k), k, dw, accumulate);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace qlora
