// 8-bit MFMA GEMM with block scales (the 8-bit layer's forward and dX).
//
//   out[m, j] = RN16( sum_c 2^(sa[m, c/128] + sf[j/128, c/128]) a[m, c] f[j, c]
//                     + sum_x split[m, x] fx[j, x] )
//
// a, f: E4M3 rows along the contraction (fp8.h), padded to 128 with zeros;
// split / fx: the 16-bit low-rank columns [hi | lo] of s T (or s U; about 16 bits
// of each in bf16, 22 of the row's largest in fp16) against [B | B] (or A^T
// twice), added to the same fp32 accumulators, so the output is rounded once.
// The 8-bit products reach the accumulators in the sums that fp8.h describes.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies E4M3 at twice the 16-bit rate
// and applies both operands' power-of-two scales inside the instruction, so
// block scaling costs no vector work. A 128-deep step of 256 rows is 32 KB,
// the same bytes as a 64-deep 16-bit step, and its 16 MFMAs per wave take the
// same 1024 cycles as the 32 of such a step: tile shape, LDS swizzle, copies
// and buffer rotation are those of the 16-bit GEMM (gemm_tile.h), with the
// activation tile in two buffers and the weight tile in three, and the rate
// doubles because each byte carries a whole element.
// Scales: one 32-bit load per lane and step brings the bytes of the wave's
// four 32-row activation blocks, picked by the instruction's byte select; the
// weight's byte is the same for the wave's 64 columns.
#include "fp8.h"
#include "gemm_tile.h"
#include "kernels.h"

namespace qlora {

namespace {

using namespace gt;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

struct F8Args {
  const uint8_t* act;   // [M, lda] codes
  const uint8_t* as;    // scale words [lda / 128][ceil(M / 128)][32]
  int64_t M, lda;
  const uint16_t* act_x;  // [M, kx] low-rank split columns
  int kx;
  const float* row_scale;  // fp16: what the split columns of each row were divided by (rows up to a multiple of 256)
  const uint8_t* f;     // [nout, ldf] codes; kNN: [kc, ldf]
  int64_t ldf, f_rows;
  const uint8_t* fs;    // scale byte of (output block, contraction block) at ob * fs_o + cb * fs_c
  int64_t fs_o, fs_c, fs_bytes;
  int64_t nout;
  const uint16_t* fx;   // [nout, kx]
  uint16_t* out;        // [M, nout]
  // whole tiles [0, full), then `tail` tiles split `splits` ways along the
  // contraction into fp32 partial tiles (as the 16-bit GEMM)
  float* part;
  int64_t full, tail;
  int splits;
};

constexpr int kCopies = 32 / kWaves;  // 1 KB copies per wave and operand tile

struct Rows {
  u32x4 a, f;  // this lane's byte offsets for its four copies of each operand
};

__device__ __forceinline__ void issue4(const i32x4& rs, const u32x4& off, int soff, char* dst) {
#pragma unroll
  for (int i = 0; i < kCopies; ++i) copy16(rs, off[i], soff, dst + i * 1024);
}

// Operand fragments of one 64-deep substep: 32 bytes per lane and 32-row
// block. The two 16-byte pieces are those of the 16-bit kernel's substeps
// 2 kk and 2 kk + 1 (conflict-free); both operands permute the contraction
// the same way, and a block of 128 shares its scale. A row block's registers
// are refilled as soon as its two MFMAs are issued; only the weight's are
// double (a second set of all six took 50 spilled registers; this one spills
// 11 in the bf16 forward, 1 in fp16, none in dX).
struct Frags {
  i32x8 a[kTM], b[2][kTN];  // b by substep parity
};

__device__ __forceinline__ i32x8 frag32(const char* T, int rb, int kk, int lane) {
  const u32x4 lo = *reinterpret_cast<const u32x4*>(T + swz(rb + (lane & 31), 4 * kk + (lane >> 5)));
  const u32x4 hi = *reinterpret_cast<const u32x4*>(T + swz(rb + (lane & 31), 4 * kk + 2 + (lane >> 5)));
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// The weight stored along its outputs (kNN; a forward's weight read for dX):
// its tile is 128 contraction rows of 256 output columns, and the same 32
// bytes of a column come back through four transposing reads of 8 rows: in
// every 16-lane group lane i addresses row base + i / 2, bytes 8 (i % 2) .. +7
// of the group's 16 columns, and receives column i of the 8 rows. Chunk c of
// row r lies at c ^ 2 (r & 7), so the 8 rows of two neighbouring groups fall
// on distinct banks. (dX of 4096 x 8192 x 22016, same box: 612 us; the weight
// transposed first and read along its rows 622 + 84.)
__device__ __forceinline__ int nn_key(int row) { return 2 * (row & 7); }

__device__ __forceinline__ i32x8 frag32_nn(const char* T, int cb, int kk, int lane) {
  const int i = lane & 15;
  const int chunk = (cb >> 4) + ((lane >> 4) & 1);
  const int row = 64 * kk + 16 * (lane >> 5) + (i >> 1);
  const char* const p = T + row * kBN + ((chunk ^ nn_key(row)) << 4) + 8 * (i & 1);  // (rows 8 apart share the key)
  typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
  const i32x2 v0 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(p));
  const i32x2 v1 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(p + 8 * kBN));
  const i32x2 v2 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(p + 32 * kBN));
  const i32x2 v3 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(p + 40 * kBN));
  return i32x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

struct Scales {
  uint32_t a, b;
};

// acc[I][*] += row block I of substep kk (the byte select is an immediate)
template <int I>
__device__ __forceinline__ void mfma_row(f32x16 (&acc)[kTM][kTN], const Frags& f, int kk, const Scales& s) {
#pragma unroll
  for (int j = 0; j < kTN; ++j)
    acc[I][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.a[I], f.b[kk][j], acc[I][j], 0, 0, I, (int)s.a, 0,
                                                                (int)s.b);
  __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ void read_a(Frags& f, const char* Ac, int wm0, int i, int kk, int lane) {
  f.a[i] = frag32(Ac, wm0 + 32 * i, kk, lane);
  __builtin_amdgcn_sched_barrier(0);
}

template <bool kNN>
__device__ __forceinline__ void read_b(Frags& f, const char* Bc, int wn0, int kk, int lane) {
#pragma unroll
  for (int j = 0; j < kTN; ++j) {
    if constexpr (kNN)
      f.b[kk][j] = frag32_nn(Bc, wn0 + 32 * j, kk, lane);
    else
      f.b[kk][j] = frag32(Bc, wn0 + 32 * j, kk, lane);
  }
  __builtin_amdgcn_sched_barrier(0);
}

struct Rsrc {
  i32x4 act, as, f, fs;
  uint32_t as_off, as_step, fs_off, fs_step;  // scale offsets: this lane's word, bytes per step
  uint32_t f_step;                            // weight bytes per step
};

__device__ __forceinline__ void load_scales(const Rsrc& rs, int step, Scales& s) {
  s.a = raw_buffer_load_u32(rs.as, (int)rs.as_off, (int)((uint32_t)step * rs.as_step), 0);
  s.b = raw_buffer_load_u8(rs.fs, (int)rs.fs_off, (int)((uint32_t)step * rs.fs_step), 0);
}

// One 128-deep step: MFMAs on (Ac, Bc) while the activation copies of step +
// 1 fill An and the weight copies of step + 2 fill Bn2. The fragments of the
// next substep are read between the MFMAs of the current one. The barrier
// (the copies of step + 1 have landed; the weight copies of step + 2 may be
// in flight) stands after the first row block of the second substep: its MFMAs
// hide the last reads before the barrier, those after it the reads of step +
// 1's first substep from (An, Bn1). (4096 x 8192 x 22016, same box: 625 us; one
// block earlier 636, one later 647, two later 658.) The scales of step + 1 are
// loaded before the copies, so the same wait covers them.
template <bool kNN>
__device__ __forceinline__ void f8_step(const Rsrc& rs, const Rows& p, int step, int nk, int wave,
                                        const char* __restrict__ Ac, const char* __restrict__ Bc,
                                        char* __restrict__ An, const char* __restrict__ Bn1, char* __restrict__ Bn2,
                                        f32x16 (&acc)[kTM][kTN], Frags& f, const Scales& cur, Scales& nxt) {
  const int lane = threadIdx.x & 63;
  const int wm0 = (wave >> 2) * 128, wn0 = (wave & 3) * 64;
  const int s1 = step + 1 < nk ? step + 1 : nk - 1;
  const int s2 = step + 2 < nk ? step + 2 : nk - 1;
  load_scales(rs, s1, nxt);
  __builtin_amdgcn_sched_barrier(0);
  issue4(rs.act, p.a, s1 * 128, An + wave * kCopies * 1024);
  issue4(rs.f, p.f, (int)((uint32_t)s2 * rs.f_step), Bn2 + wave * kCopies * 1024);
  __builtin_amdgcn_sched_barrier(0);
  mfma_row<0>(acc, f, 0, cur);
  read_b<kNN>(f, Bc, wn0, 1, lane);
  read_a(f, Ac, wm0, 0, 1, lane);
  mfma_row<1>(acc, f, 0, cur);
  read_a(f, Ac, wm0, 1, 1, lane);
  mfma_row<2>(acc, f, 0, cur);
  read_a(f, Ac, wm0, 2, 1, lane);
  mfma_row<3>(acc, f, 0, cur);
  read_a(f, Ac, wm0, 3, 1, lane);
  mfma_row<0>(acc, f, 1, cur);
  step_barrier<kCopies>();
  __builtin_amdgcn_sched_barrier(0);
  read_b<kNN>(f, Bn1, wn0, 0, lane);
  read_a(f, An, wm0, 0, 0, lane);
  mfma_row<1>(acc, f, 1, cur);
  read_a(f, An, wm0, 1, 0, lane);
  mfma_row<2>(acc, f, 1, cur);
  read_a(f, An, wm0, 2, 0, lane);
  mfma_row<3>(acc, f, 1, cur);
  read_a(f, An, wm0, 3, 0, lane);
}

// First copies: step sbeg of both operands and the weight of step sbeg + 1
// (restrict pointers, so the compiler can tell them from the loop's reads).
__device__ __forceinline__ void f8_prologue(const Rsrc& rs, const Rows& p, int sbeg, int nk, int wave,
                                            char* __restrict__ A0, char* __restrict__ B0, char* __restrict__ B1,
                                            Scales& s) {
  load_scales(rs, sbeg, s);
  issue4(rs.act, p.a, sbeg * 128, A0 + wave * kCopies * 1024);
  issue4(rs.f, p.f, (int)((uint32_t)sbeg * rs.f_step), B0 + wave * kCopies * 1024);
  issue4(rs.f, p.f, (int)((uint32_t)(sbeg + 1 < nk ? sbeg + 1 : nk - 1) * rs.f_step), B1 + wave * kCopies * 1024);
  step_barrier<kCopies>();
}

template <bool kF16, bool kNN>
__global__ __launch_bounds__(kThreads) void gemm_fp8_kernel(F8Args a) {
  __shared__ __attribute__((aligned(16))) char As0[kTileBytes];
  __shared__ __attribute__((aligned(16))) char As1[kTileBytes];
  __shared__ __attribute__((aligned(16))) char Bs0[kTileBytes];
  __shared__ __attribute__((aligned(16))) char Bs1[kTileBytes];
  __shared__ __attribute__((aligned(16))) char Bs2[kTileBytes];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm0 = (wave >> 2) * 128, wn0 = (wave & 3) * 64;
  const int64_t mt = cdiv(a.M, (int64_t)kBM), nt = cdiv(a.nout, (int64_t)kBN);
  const int b = (int)blockIdx.x;
  const bool whole = b < a.full;
  const int unit = whole ? 0 : b - (int)a.full;
  const int tail_i = whole ? 0 : __builtin_amdgcn_readfirstlane(unit % (int)a.tail);
  const int split = whole ? 0 : __builtin_amdgcn_readfirstlane(unit / (int)a.tail);
  int64_t tm, tn;
  tile_of(tm, tn, mt, nt, whole ? (int64_t)b : a.full + tail_i);
  const int64_t m0 = tm * kBM, n0 = tn * kBN;
  const int nk_all = (int)(a.lda / kF8Block);
  const int chunk = whole ? nk_all : __builtin_amdgcn_readfirstlane((nk_all + a.splits - 1) / a.splits);
  const int sbeg = split * chunk;
  const int nk = sbeg + chunk < nk_all ? sbeg + chunk : nk_all;  // exclusive end

  f32x16 acc[kTM][kTN];
#pragma unroll
  for (int i = 0; i < kTM; ++i)
#pragma unroll
    for (int j = 0; j < kTN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  // Low-rank columns first (1 - 4 steps of 64 16-bit columns, the first range only)
  if (sbeg == 0) {
    for (int x = 0; x < a.kx; x += kBK) {
      issue_tile_lds(a.act_x, a.kx, a.M, m0, a.kx, x, As0);
      issue_tile_lds(a.fx, a.kx, a.nout, n0, a.kx, x, Bs0);
      step_barrier<0>();
#pragma unroll
      for (int kk = 0; kk < kBK / 16; ++kk) {
        bf16x8 af[kTM], bfr[kTN];
#pragma unroll
        for (int i = 0; i < kTM; ++i) af[i] = tile_frag(As0, wm0 + i * 32, kk, lane);
#pragma unroll
        for (int j = 0; j < kTN; ++j) bfr[j] = tile_frag(Bs0, wn0 + j * 32, kk, lane);
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
          for (int j = 0; j < kTN; ++j) acc[i][j] = mfma32<kF16>(af[i], bfr[j], acc[i][j]);
      }
      __syncthreads();  // every wave's reads done before the next copies land
    }
    if constexpr (kF16) {
      if (a.kx > 0) scale_rows(acc, a.row_scale, 0, m0 + wm0, lane);
    }
  }

  {
    Rows p;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int row = (wave * kCopies + i) * 8 + (lane >> 3);
      const int lc = (lane & 7) ^ swz_key(row);
      const int64_t m = m0 + row < a.M ? m0 + row : a.M - 1;  // rows past the end repeat the last (not stored)
      const int64_t n = n0 + row < a.nout ? n0 + row : a.nout - 1;
      p.a[i] = (uint32_t)(m * a.lda + 16 * lc);
      if constexpr (kNN) {
        // columns past nout read other data (their outputs are not stored),
        // rows past the end zeros (range check)
        const int r = (wave * kCopies + i) * 4 + (lane >> 4);
        p.f[i] = (uint32_t)(r * a.ldf + n0 + 16 * ((lane & 15) ^ nn_key(r)));
      } else {
        p.f[i] = (uint32_t)(n * a.ldf + 16 * lc);
      }
    }
    Rsrc rs;
    const int64_t mt128 = cdiv(a.M, (int64_t)kF8Block);
    rs.act = make_rsrc(a.act, a.M * a.lda);
    rs.f = make_rsrc(a.f, a.f_rows * a.ldf);
    rs.f_step = kNN ? (uint32_t)(128 * a.ldf) : 128u;
    rs.as = make_rsrc(a.as, (int64_t)nk_all * mt128 * 128);
    rs.fs = make_rsrc(a.fs, a.fs_bytes);
    // (row tiles past M and output blocks past nout: any in-range scale, the results are not stored)
    const int64_t t128 = (m0 + wm0) / kF8Block < mt128 ? (m0 + wm0) / kF8Block : mt128 - 1;
    const int64_t ob = (n0 + wn0 < a.nout ? n0 + wn0 : a.nout - 1) / kF8Block;
    rs.as_off = (uint32_t)(t128 * 128 + 4 * (lane & 31));
    rs.as_step = (uint32_t)(mt128 * 128);
    rs.fs_off = (uint32_t)(ob * a.fs_o);
    rs.fs_step = (uint32_t)a.fs_c;
    Scales s0, s1;
    Frags f;
    f8_prologue(rs, p, sbeg, nk, wave, As0, Bs0, Bs1, s0);
    read_b<kNN>(f, Bs0, wn0, 0, lane);
#pragma unroll
    for (int i = 0; i < kTM; ++i) read_a(f, As0, wm0, i, 0, lane);
    f8_step<kNN>(rs, p, sbeg, nk, wave, As0, Bs0, As1, Bs1, Bs2, acc, f, s0, s1);
    int s = sbeg + 1;
    for (; s + 6 <= nk; s += 6) {
      f8_step<kNN>(rs, p, s, nk, wave, As1, Bs1, As0, Bs2, Bs0, acc, f, s1, s0);
      f8_step<kNN>(rs, p, s + 1, nk, wave, As0, Bs2, As1, Bs0, Bs1, acc, f, s0, s1);
      f8_step<kNN>(rs, p, s + 2, nk, wave, As1, Bs0, As0, Bs1, Bs2, acc, f, s1, s0);
      f8_step<kNN>(rs, p, s + 3, nk, wave, As0, Bs1, As1, Bs2, Bs0, acc, f, s0, s1);
      f8_step<kNN>(rs, p, s + 4, nk, wave, As1, Bs2, As0, Bs0, Bs1, acc, f, s1, s0);
      f8_step<kNN>(rs, p, s + 5, nk, wave, As0, Bs0, As1, Bs1, Bs2, acc, f, s0, s1);
    }
    const int rem = nk - s;
    if (rem > 0) f8_step<kNN>(rs, p, s, nk, wave, As1, Bs1, As0, Bs2, Bs0, acc, f, s1, s0);
    if (rem > 1) f8_step<kNN>(rs, p, s + 1, nk, wave, As0, Bs2, As1, Bs0, Bs1, acc, f, s0, s1);
    if (rem > 2) f8_step<kNN>(rs, p, s + 2, nk, wave, As1, Bs0, As0, Bs1, Bs2, acc, f, s1, s0);
    if (rem > 3) f8_step<kNN>(rs, p, s + 3, nk, wave, As0, Bs1, As1, Bs2, Bs0, acc, f, s0, s1);
    if (rem > 4) f8_step<kNN>(rs, p, s + 4, nk, wave, As1, Bs2, As0, Bs0, Bs1, acc, f, s1, s0);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<0>());
    __syncthreads();
  }

  if (!whole) {
    float* const pp = a.part + ((int64_t)split * a.tail + tail_i) * (kBM * kBN);
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
      for (int j = 0; j < kTN; ++j) {
        const int c = wn0 + j * 32 + (lane & 31);
        if (n0 + c >= a.nout) continue;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int rr = wm0 + i * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
          if (m0 + rr < a.M) pp[rr * kBN + c] = acc[i][j][v];
        }
      }
    return;
  }
  char* const buf = wave < 4 ? (wave < 2 ? As0 : As1) : (wave < 6 ? Bs0 : Bs1);
  store_staged<kF16>(acc, reinterpret_cast<uint16_t*>(buf + (wave & 1) * 16384), a.out, a.M, a.nout, m0 + wm0, n0 + wn0,
                     lane);
}

}  // namespace

// 32-bit offsets (kNN reads up to a tile's width past the operand's end, where the range check has to see it)
bool gemm_fp8_offsets_fit(int64_t M, int64_t kc, int kx, int64_t nout, bool nn) {
  const int64_t lim = (int64_t)1 << 32;
  const int64_t fb = nn ? f8_pad(kc) * f8_pad(nout) + kBN : nout * f8_pad(kc);
  return M * f8_pad(kc) < lim && fb < lim && M * (int64_t)kx * 2 < lim && nout * (int64_t)kx * 2 < lim;
}

size_t gemm_fp8_ws_bytes(int64_t M, int64_t kc, int64_t nout) {
  const GemmSplit p = gemm_split_plan(M, nout, f8_pad(kc) / kF8Block);
  return p.splits > 1 ? align256((size_t)p.splits * (size_t)p.tail * kBM * kBN * 4) : 0;
}

hipError_t launch_gemm_fp8(const uint8_t* act, const uint8_t* as, int64_t M, int64_t kc, const uint16_t* split, int kx,
                           const float* row_scale,
                           const uint8_t* f, const uint8_t* fs, int64_t fs_o, int64_t fs_c, int64_t fs_bytes,
                           const uint16_t* fx, int64_t nout, uint16_t* out, float* part, hipStream_t stream, bool f16,
                           bool nn) {
  if (f16 && kx > 0 && row_scale == nullptr) return hipErrorInvalidValue;
  F8Args a{};
  a.row_scale = row_scale;
  a.act = act; a.as = as; a.M = M; a.lda = f8_pad(kc);
  a.act_x = split; a.kx = kx;
  a.f = f; a.fs = fs; a.fs_o = fs_o; a.fs_c = fs_c; a.fs_bytes = fs_bytes;
  a.ldf = nn ? f8_pad(nout) : a.lda; a.f_rows = nn ? kc : nout;
  a.nout = nout; a.fx = fx; a.out = out;
  const GemmSplit sp = gemm_split_plan(M, nout, a.lda / kF8Block);
  a.full = sp.full; a.tail = sp.tail; a.splits = sp.splits;
  a.part = part;
  if (a.splits > 1 && part == nullptr) return hipErrorInvalidValue;
  const dim3 grid((unsigned)(a.full + a.tail * a.splits));
#define QLORA_GEMM8(H, NN) gemm_fp8_kernel<H, NN><<<grid, kThreads, 0, stream>>>(a)
  if (f16 && nn) QLORA_GEMM8(true, true);
  else if (f16) QLORA_GEMM8(true, false);
  else if (nn) QLORA_GEMM8(false, true);
  else QLORA_GEMM8(false, false);
#undef QLORA_GEMM8
  if (a.splits > 1) return launch_gemm_reduce(part, sp, M, nout, out, stream, f16);
  return hipGetLastError();
}

}  // namespace qlora
