// 8-bit layer for few tokens: one pass over the weight's codes for each 16 of
// them, or 32.
//
//   Y = RN16( X8 W8^T + s T B^T )
//
// Bound by HBM: every code byte serves at most 32 tokens. fp8_prep_kernel has
// encoded X into the operand order of v_mfma_scale_f32_16x16x128_f8f6f4 (per
// 128-column block and lane: 32 bytes of one token row, zeros past M), so that
// X is read in runs of 1 KB, and left T = X A^T in a few partials, which each
// workgroup adds while its first codes are on the way (a launch less).
// A workgroup owns 16 kT weight rows; its 8 waves take the 128-column blocks
// in turn, so neighbouring waves read neighbouring lines of the same rows.
// Codes go from memory straight into LDS, eight neighbouring lanes a 128-byte
// line, into a ring of three blocks per wave (one multiplied, two in flight), and
// from there in operand order (a lane takes 32 consecutive bytes of one row).
// Loaded in operand order they cost a cache access per lane: 52 us for 8192 x
// 28672 at one token.
// Partial sums of the waves are added in wave order through LDS, the low-rank
// term is added in fp32, and Y is rounded once. What a sum of 8 products holds
// inside the instruction is said in fp8.h.
#include "fp8.h"
#include "kernels.h"

namespace qlora {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kGvWaves = 8;
constexpr int kMaxR = 128;  // largest rank

__device__ __forceinline__ i32x8 join(const u32x4& lo, const u32x4& hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// Row r of a tile keeps its 16-byte segment s at s ^ swz(r): the 16 rows that
// one cycle reads lie on distinct banks.
__device__ __forceinline__ int row_swz(int r) { return (r ^ (r >> 3)) & 7; }

template <int kMT>
struct Block {
  u32x4 x[kMT][2];
  uint32_t xs[kMT], ws;
};

// kRows: the activations as codes [M, kp] and scales [M, kp / 128] of each row
// (the lanes of a row's 128 columns read one line of it; rows from M on repeat
// the last, their sums are not stored) instead of operand order.
// kMT: token tiles of 16 that a workgroup multiplies with each code it reads (two
// take 124 registers a lane: at more than 128 a compute unit would hold one
// workgroup, 11008 x 4096 at 64 tokens 31 us against 25); the grid's second dimension
// is groups of kMT tiles.
template <int kT, int kMT, bool kF16, bool kRows>
__global__ __launch_bounds__(64 * kGvWaves) void gemv_fp8_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ wscale, int64_t N,
                                                                 int64_t kp, const uint8_t* __restrict__ Xq,
                                                                 const uint8_t* __restrict__ Xs, int64_t M,
                                                                 const float* __restrict__ T, int parts,
                                                                 const uint16_t* __restrict__ B, int r, float scale,
                                                                 uint16_t* __restrict__ Y, float* __restrict__ T_save) {
  constexpr int NT = 16 * kT;
  constexpr int kSlot = kT * 2048;  // one wave's codes of one block
  // three arrays, so that the compiler can tell the one being read from those
  // being filled
  __shared__ __attribute__((aligned(16))) char ring0[kGvWaves * kSlot];
  __shared__ __attribute__((aligned(16))) char ring1[kGvWaves * kSlot];
  __shared__ __attribute__((aligned(16))) char ring2[kGvWaves * kSlot];
  static_assert(kMT == 1 || !kRows, "tokens by row: one tile");
  __shared__ float lred[kT][16][16];
  __shared__ __attribute__((aligned(16))) float Ts[16 * kMT * (kMaxR + 4)];  // T [the group's tokens][r]
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * NT;
  const int nb = (int)(kp / kF8Block);
  const int64_t rows = N - n0 < NT ? N - n0 : NT;
  const int64_t mg = (int64_t)blockIdx.y * 16 * kMT;  // the group's first token
  const int Ml = (int)(M - mg < 16 * kMT ? M - mg : 16 * kMT);
  const int tiles = (Ml + 15) / 16;
  // this workgroup's rows (those past N read as zero and are not stored)
  const i32x4 wr = make_rsrc(codes + n0 * kp, rows * kp);
  const i32x4 sr = make_rsrc(wscale + (n0 / kF8Block) * nb, nb);
  // (token tiles past the last read as zero)
  const i32x4 xr = make_rsrc(Xq + (kRows ? 0 : mg / 16 * nb * 2048), kRows ? M * kp : (int64_t)tiles * nb * 2048);
  const i32x4 xsr = make_rsrc(Xs + (kRows ? 0 : mg / 16 * nb * 16), kRows ? M * nb : (int64_t)tiles * nb * 16);
  const int xm = (lane & 15) < M ? (lane & 15) : (int)M - 1;
  const int xoff = kRows ? (int)(xm * kp) + 32 * (lane >> 4) : lane * 32;
  const int xsoff = kRows ? xm * nb : lane & 15;
  // copy h of tile i: lane l fills row 8 h + l / 8, position l % 8
  uint32_t woff[kT][2];
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 8 * h + (lane >> 3);
      woff[i][h] = (uint32_t)((16 * i + row) * kp + 16 * ((lane & 7) ^ row_swz(row)));
    }
  const int rd = (lane & 15) * 128 + 16 * ((2 * (lane >> 4)) ^ row_swz(lane & 15));

  const int cnt = wave < nb ? (nb - 1 - wave) / kGvWaves + 1 : 0;
  auto issue = [&](int j, char* R, Block<kMT>& b) {
    const int kb = wave + kGvWaves * (j < cnt ? j : cnt - 1);  // past the range: the last block again
    char* const dst = R + wave * kSlot;
#pragma unroll
    for (int i = 0; i < kT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) copy16(wr, woff[i][h], kb * kF8Block, dst + i * 2048 + h * 1024);
#pragma unroll
    for (int q = 0; q < kMT; ++q) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        b.x[q][h] = raw_buffer_load_b128(xr, xoff + 16 * h, kRows ? kb * kF8Block : (q * nb + kb) * 2048, 0);
      b.xs[q] = raw_buffer_load_u8(xsr, xsoff, kRows ? kb : (q * nb + kb) * 16, 0);
    }
    b.ws = raw_buffer_load_u8(sr, 0, kb, 0);
  };
  f32x4 acc[kT][kMT];
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int q = 0; q < kMT; ++q) acc[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const char* R, const Block<kMT>& b) {
    const char* const src = R + wave * kSlot + rd;
    const char* const src2 = R + wave * kSlot + (rd ^ 16);
#pragma unroll
    for (int i = 0; i < kT; ++i) {
      const i32x8 w =
          join(*reinterpret_cast<const u32x4*>(src + i * 2048), *reinterpret_cast<const u32x4*>(src2 + i * 2048));
#pragma unroll
      for (int q = 0; q < kMT; ++q)
        acc[i][q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(b.x[q][0], b.x[q][1]), w, acc[i][q], 0, 0, 0,
                                                                     (int)b.xs[q], 0, (int)b.ws);
    }
  };
  Block<kMT> s0, s1, s2;
  if (cnt > 0) {
    issue(0, ring0, s0);
    issue(1, ring1, s1);
  }
  // B of the tiles' rows, all of it under way before the codes are waited for
  // (loaded rank by rank in the loop that uses it, at rank 64 the epilogue took
  // longer than the codes: 11008 x 4096 at 16 tokens 22.5 us). One test for r = 0: the
  // loop's own, a branch for each load, cost a call without an adapter 0.1 - 0.2 us of 13.
  uint32_t bq[kMaxR / 4];
  const i32x4 br = make_rsrc(B, 2 * N * r);
  if (r > 0 && wave < kT) {
    const int64_t n = n0 + wave * 16 + (lane & 15);
    const int boff = n < N ? (int)(2 * (n * r + (lane >> 4))) : -1;  // (past every row: zero)
#pragma unroll
    for (int i = 0; i < kMaxR / 4; ++i)
      if (4 * i < r) bq[i] = raw_buffer_load_u16(br, boff, 8 * i, 0);
  }
  // T into LDS: added up already, four values a load, or partials, added here. Rows
  // of r + 4 where r is a multiple of 4 (the 16 rows that one instruction reads on
  // distinct banks).
  const int pitch = r % 4 == 0 ? r + 4 : r;
  const float* const src = T + mg * r;  // (r times a multiple of 16 floats: as aligned as T)
  if (parts == 1) {
    const int quads = Ml * r / 4;
    for (int o = t; o < quads; o += 64 * kGvWaves) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(src + 4 * o);
#pragma unroll
      for (int e = 0; e < 4; ++e) Ts[(4 * o + e) / r * pitch + (4 * o + e) % r] = v[e];
    }
    for (int o = 4 * quads + t; o < Ml * r; o += 64 * kGvWaves) Ts[o / r * pitch + o % r] = src[o];
    if (T_save != nullptr && blockIdx.x == 0) {
      for (int o = t; o < Ml * r; o += 64 * kGvWaves) T_save[mg * r + o] = src[o];
    }
  }
  if (parts > 1) {
    for (int o = t; o < Ml * r; o += 64 * kGvWaves) {
      float s = 0.0f;
      for (int p0 = 0; p0 < parts; p0 += 8) {  // eight loads in flight, added in order
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = src[(int64_t)(p0 + e < parts ? p0 + e : parts - 1) * M * r + o];
#pragma unroll
        for (int e = 0; e < 8; ++e) s += p0 + e < parts ? v[e] : 0.0f;
      }
      Ts[o / r * pitch + o % r] = s;
      if (T_save != nullptr && blockIdx.x == 0) T_save[mg * r + o] = s;
    }
  }
  if (cnt > 0) {
    // whole groups of three with no exit inside (an exit leaves a path on which
    // the compiler waits for every load in flight)
    int j = 0;
    for (; j + 3 <= cnt; j += 3) {
      issue(j + 2, ring2, s2);
      __builtin_amdgcn_sched_barrier(0);
      compute(ring0, s0);
      __builtin_amdgcn_sched_barrier(0);
      issue(j + 3, ring0, s0);
      __builtin_amdgcn_sched_barrier(0);
      compute(ring1, s1);
      __builtin_amdgcn_sched_barrier(0);
      issue(j + 4, ring1, s1);
      __builtin_amdgcn_sched_barrier(0);
      compute(ring2, s2);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (j < cnt) compute(ring0, s0);
    if (j + 1 < cnt) compute(ring1, s1);
  }
  // copies past the range may still be landing: done before the ring is reused
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  float(*const red)[kT][16][16] = reinterpret_cast<float(*)[kT][16][16]>(ring0);  // [wave]
  static_assert(sizeof(float) * kGvWaves * kT * 256 <= kGvWaves * kSlot, "partials fit the ring");

#pragma unroll
  for (int q = 0; q < kMT; ++q) {
    if (q > 0) __syncthreads();  // the last tile's sums are read
    // D[m][n]: lane -> n = lane % 16, m = 4 (lane / 16) + v
#pragma unroll
    for (int i = 0; i < kT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wave][i][4 * (lane >> 4) + v][lane & 15] = acc[i][q][v];
    if (r > 0 && wave < kT) {
      // L[m][n] = sum_j T[m][j] B[n][j], 4 ranks per fp32 MFMA (T and B exact)
      const int i = wave;
      f32x4 l = f32x4{0.f, 0.f, 0.f, 0.f};
      const int m = 16 * q + (lane & 15);
#pragma unroll
      for (int e = 0; e < kMaxR / 4; ++e) {
        if (4 * e >= r) break;
        const int j = 4 * e + (lane >> 4);
        const float a = (m < Ml && j < r) ? Ts[m * pitch + j] : 0.0f;
        const float b = j < r ? from16<kF16>(bq[e]) : 0.0f;
        l = __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, l, 0, 0, 0);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) lred[i][4 * (lane >> 4) + v][lane & 15] = l[v];
    }
    __syncthreads();
    for (int o = t; o < 16 * NT; o += 64 * kGvWaves) {
      const int m = o / NT, nl = o % NT;
      const int64_t n = n0 + nl;
      if (16 * q + m >= Ml || n >= N) continue;
      const int i = nl >> 4, nc = nl & 15;
      float y = red[0][i][m][nc];
#pragma unroll
      for (int w = 1; w < kGvWaves; ++w) y += red[w][i][m][nc];  // in wave order
      if (r > 0) y = fmaf(scale, lred[i][m][nc], y);
      Y[(mg + 16 * q + m) * N + n] = to16<kF16>(y);
    }
  }
}

}  // namespace

size_t fp8_gemv_codes_bytes(int64_t k, int64_t M) {
  return (size_t)cdiv(M, (int64_t)16) * (size_t)(f8_pad(k) / kF8Block) * 2048;
}
size_t fp8_gemv_scale_bytes(int64_t k, int64_t M) {
  return (size_t)cdiv(M, (int64_t)16) * (size_t)(f8_pad(k) / kF8Block) * 16;
}

hipError_t launch_fp8_gemv(const Fp8View& w, const uint8_t* xq, const uint8_t* xs, bool rows, int64_t M, const float* T,
                           int parts, const uint16_t* B, int r, float scale, uint16_t* Y, float* T_save,
                           hipStream_t stream, bool f16) {
  if (M < 1 || M > kGemvMostTokens || (rows && M > 16)) return hipErrorInvalidValue;
#define QLORA_GV8M(KT, MT, H, R)                                                                                   \
  gemv_fp8_kernel<KT, MT, H, R>                                                                                    \
      <<<dim3((unsigned)cdiv(w.n, (int64_t)(16 * KT)), (unsigned)cdiv(M, (int64_t)(16 * MT))), 64 * kGvWaves, 0,   \
         stream>>>(w.codes, w.scale, w.n, f8_pad(w.k), xq, xs, M, T, parts, B, r, scale, Y, T_save)
#define QLORA_GV8(KT, H)                          \
  {                                               \
    if (M > 16) QLORA_GV8M(KT, 2, H, false);      \
    else if (rows) QLORA_GV8M(KT, 1, H, true);    \
    else QLORA_GV8M(KT, 1, H, false);             \
  }
  // One tile of rows takes 57 KB of LDS (two workgroups on a CU), two tiles 106
  // (one). Two where that gives a CU at most one workgroup and one tile would give
  // some CUs two (4097 to 8192 rows): every CU then reads alone and to the end.
  // One token, encode included, one against two tiles: 4200 x 28672 46 and 38 us,
  // 8192 x 28672 55 and 50, 7168 x 4096 13.0 and 12.1, 8192 x 8192 18.3 and 18.9.
  // Fewer rows leave CUs idle with two tiles (4096 x 28672 31 and 40 us), more
  // start a second round of them (8200 x 8192 20 and 22, 11008 x 8192 25 and 27).
  // (One token that comes encoded, r = 0: 8192 x 8192 13.5 and 17.0, 8192 x 28672 41 and 43.)
  // 17 to 32 tokens, encoded, r = 64: 4200 x 4096 19.6 and 18.1, 5120 x 13824 41.8 and
  // 34.9, 8192 x 28672 77 and 61. From 33 on a second group of token tiles gives a CU a
  // second workgroup either way, and neither is better throughout: 33 tokens, r = 64,
  // 4200 x 4096 23.4 and 24.7, 7168 x 4096 26.4 and 25.3, 8192 x 4096 26.8 both, 8192 x
  // 8192 40.2 and 44.3.
  constexpr int64_t kCus = 256;
  if (w.n > 16 * kCus && w.n <= 32 * kCus) {
    if (f16) QLORA_GV8(2, true) else QLORA_GV8(2, false)
  } else {
    if (f16) QLORA_GV8(1, true) else QLORA_GV8(1, false)
  }
#undef QLORA_GV8
#undef QLORA_GV8M
  return hipGetLastError();
}

}  // namespace qlora
