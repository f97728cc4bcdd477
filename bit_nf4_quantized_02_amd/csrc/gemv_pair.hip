// The gated feed-forward block's few-token form (M <= 16):
//
//   G = X Wg'^T + s Tg Bg^T,  U = X Wu'^T + s Tu Bu^T,  H = RN16( silu(G) U )
//
// from the unrounded fp32 G and U, in three launches: the projections (and from
// 5 tokens X in operand order), their low-rank products L = s T B^T over the
// n outputs, and one pass over both weights' codes.
//
// The pass expands codes as the plain few-token kernel does (gemv_nf4.hip: a
// ring of code chunks in LDS filled by direct copies, levels of two weights per
// table read, v_mfma_f32_16x16x32 with the weight as B operand), with 16 gate
// rows as one tile and the same 16 up rows as the other, so that X is read once
// for both. It is persistent: one workgroup of eight waves per CU takes row
// groups in turn, the table is built once and the ring runs on from one group
// into the next, whose first chunks are in flight while the last group's sums
// are joined. Bound by the expansion (about 3 vector operations per weight and
// one LDS read per two) as much as by HBM. (28672 x 8192, one token: 63 us,
// 3.9 TB/s of codes and scales; 11008 x 4096, 16 fp16 tokens: 22. A workgroup
// of four waves for each row group, two on a CU: 77 and 29.)
#include "common.h"
#include "gemv_nf4.h"
#include "kernels.h"

namespace qlora {

namespace {

// X [M, K] for few tokens in operand order (xp not
// NULL), and the projections X Ag^T, X Au^T as partials [range][2][M][r]. A
// wave takes 128-column blocks in turn: 16 neighbouring lanes load 256 bytes of
// a row, which pass through the wave's own LDS into the A operand of
// v_mfma_f32_16x16x32; the workgroup's four waves are added in wave order. The
// blocks cover whole 256-column chunks (zeros past K), as the GEMV reads them.
template <int kRP, bool kF16>
__global__ __launch_bounds__(256) void gemv_prep_kernel(const uint16_t* __restrict__ X, int64_t M, int64_t K, int nb,
                                                        const uint16_t* __restrict__ Ag, const uint16_t* __restrict__ Au,
                                                        int r, int bchunk, u32x4* __restrict__ xp,
                                                        float* __restrict__ part) {
  constexpr int kTiles = kRP / 16, kTA = kTiles > 0 ? kTiles : 1;
  constexpr int kPitch = 256 + 16;
  __shared__ __attribute__((aligned(16))) char turn[4][kTiles > 0 ? 16 * kPitch : 16];
  __shared__ float red[4][16][kTiles > 0 ? kRP : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b0 = (int)blockIdx.x * bchunk, b1 = b0 + bchunk < nb ? b0 + bchunk : nb;
  const int lr = lane >> 4, lc = 8 * (lane & 15);
  f32x4 acc[2][kTA];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int t = 0; t < kTA; ++t) acc[w][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int kb = b0 + wave; kb < b1; kb += 4) {
    u32x4 x[4], q[2][kTA][4];
    // (whole blocks load without a test per lane, which would put each load
    // behind a branch that waits for it)
    const bool whole = ((int64_t)kb + 1) * 128 <= K;
    const uint16_t* const xb = X + (int64_t)kb * 128 + lc;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t m = 4 * u + lr < M ? 4 * u + lr : M - 1;
      x[u] = whole ? *reinterpret_cast<const u32x4*>(xb + m * K) : load8h<true>(X + m * K, (int64_t)kb * 128 + lc, K);
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int64_t j = 16 * t + (lane & 15) < r ? 16 * t + (lane & 15) : r - 1;  // (ranks past r: not stored)
        const int64_t c = (int64_t)kb * 128 + 32 * s + 8 * (lane >> 4);
        q[0][t][s] = whole ? *reinterpret_cast<const u32x4*>(Ag + j * K + c) : load8h<true>(Ag + j * K, c, K);
        q[1][t][s] = whole ? *reinterpret_cast<const u32x4*>(Au + j * K + c) : load8h<true>(Au + j * K, c, K);
      }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int m = 4 * u + lr;
      if (m >= M) x[u] = u32x4{0u, 0u, 0u, 0u};
      if (xp != nullptr) {
        const int c = (kb & 1) * 128 + lc;  // column of the 256-column chunk
        xp[((int64_t)(kb >> 1) * 8 + ((c >> 3) & 7)) * 64 + 16 * (c >> 6) + m] = x[u];
      }
      if constexpr (kTiles > 0) *reinterpret_cast<u32x4*>(turn[wave] + m * kPitch + 2 * lc) = x[u];
    }
    // lanes read what others wrote: the LDS keeps a wave's order, the compiler must too
    asm volatile("" ::: "memory");
#pragma unroll
    for (int s = 0; s < (kTiles > 0 ? 4 : 0); ++s) {
      const bf16x8 a = *reinterpret_cast<const bf16x8*>(turn[wave] + (lane & 15) * kPitch + 64 * s + 16 * (lane >> 4));
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) acc[w][t] = mfma16<kF16>(a, __builtin_bit_cast(bf16x8, q[w][t][s]), acc[w][t]);
    }
    asm volatile("" ::: "memory");
  }
  if constexpr (kTiles > 0) {
    for (int w = 0; w < 2; ++w) {
      __syncthreads();
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          red[wave][4 * (lane >> 4) + v][16 * t + (lane & 15)] = w == 0 ? acc[0][t][v] : acc[1][t][v];
      __syncthreads();
      for (int o = threadIdx.x; o < (int)M * r; o += 256) {
        const int m = o / r, j = o % r;
        part[(((int64_t)blockIdx.x * 2 + w) * M + m) * r + j] = red[0][m][j] + red[1][m][j] + red[2][m][j] + red[3][m][j];
      }
    }
  }
}

// L[w][m][n] = scale * sum_j T[w][m][j] Bw[n][j] from the projections' partials,
// added in order (T_save: T itself, from the first workgroup). 64 outputs of
// both weights per workgroup, one 16-output tile per wave; v_mfma_f32_16x16x4
// multiplies fp32 T and exact B, the ranks taken 8 per lane group so that a
// lane's B values are one load. (A launch of its own, 5 us: in the pass over
// the codes each row group would wait for its B rows.)
template <bool kF16>
__global__ __launch_bounds__(256) void pair_lowrank_kernel(const float* __restrict__ part, int parts, int64_t M, int r,
                                                           float scale, const uint16_t* __restrict__ Bg,
                                                           const uint16_t* __restrict__ Bu, int64_t N,
                                                           float* __restrict__ T_save, float* __restrict__ L) {
  constexpr int kPitch = 128 + 4;
  __shared__ float T[2][16][kPitch];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int steps = (r + 31) / 32, rz = steps * 32;
  const int64_t n0 = (int64_t)blockIdx.x * 64 + wave * 16;
  const int64_t n = n0 + (lane & 15);
  const int64_t nr = n < N ? n : N - 1;  // (outputs past N: not stored)
  // B first: its loads are on the way while the partials are added
  u32x4 b[2][4];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int j0 = 32 * s + 8 * (lane >> 4);
      b[w][s] = u32x4{0u, 0u, 0u, 0u};
      if (j0 < r) b[w][s] = load8h<false>((w == 0 ? Bg : Bu) + nr * r, j0, r);
    }
  // four ranks per thread, eight partials' loads together (those past the last repeat it and are not added)
  const bool vec = r % 4 == 0;
  for (int i = threadIdx.x; i < 2 * 16 * (rz / 4); i += 256) {
    const int j = 4 * (i % (rz / 4)), m = i / (rz / 4) % 16, w = i / (rz / 4) / 16;
    f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
    if (m < M && j < r) {
      const float* const src = part + ((int64_t)w * M + m) * r + j;
      const int64_t pitch = (int64_t)2 * M * r;
      for (int p0 = 0; p0 < parts; p0 += 8) {
        f32x4 x[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const float* const at = src + (p0 + p < parts ? p0 + p : parts - 1) * pitch;
          if (vec) {
            x[p] = *reinterpret_cast<const f32x4*>(at);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[p][e] = at[j + e < r ? e : 0];
          }
        }
#pragma unroll
        for (int p = 0; p < 8; ++p)
          if (p0 + p < parts) s = p0 + p == 0 ? x[p] : s + x[p];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (j + e >= r) s[e] = 0.0f;
        if (j + e < r && T_save != nullptr && blockIdx.x == 0) T_save[((int64_t)w * M + m) * r + j + e] = s[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) T[w][m][j + e] = s[e];
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    f32x4 l = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s >= steps) break;
      const int j0 = 32 * s + 8 * (lane >> 4);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        l = __builtin_amdgcn_mfma_f32_16x16x4f32(
            T[w][lane & 15][j0 + e], from16<kF16>((b[w][s][e >> 1] >> (16 * (e & 1))) & 0xFFFFu), l, 0, 0, 0);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t m = 4 * (lane >> 4) + v;
      if (m < M && n < N) L[(w * M + m) * N + n] = scale * l[v];
    }
  }
}

struct PairWeight {
  const uint8_t* codes;
  const uint8_t* code8;
  const float* s2;
  const float* mean;
  const float* codebook;
};

constexpr int kPW = 8;               // waves
constexpr int kSlot = 2 * 2048;      // a wave's codes of one chunk: 16 rows x 128 bytes of each weight
static_assert(kSlot >= 2 * 2 * 256 * 4, "the sums of two row groups fit a slot");
constexpr int64_t kPairGroups = 256;  // workgroups: one per CU

// Where the activation operand comes from: X in place; the operand-ordered copy
// Xp; up to four tokens, two loads whose 16-lane rows hold the four tokens' 32
// columns each, turned within the row to the eight fragments (rows past the
// fourth then repeat the others, and their results are not stored). The eight
// loads of the other forms keep the address units busy for twice as long as the
// codes' copies: 28672 x 8192 at 1 and 4 tokens 66 and 67 us with two loads, 69
// and 71 in place, 78 and 79 from Xp, whose zero rows are read too.
constexpr int kXPlace = 0, kXOrder = 1, kXFour = 2;

// One 256-column chunk: the lane's scale fields of both weights, its
// activation operand, and its share of L for the row group.
template <int kX>
struct PairStage {
  uint32_t c8[2];
  uint32_t s2[2];
  float l;
  u32x4 xa[kX == kXFour ? 2 : 8];
};

// Lane i of every 16-lane row receives lane (i + 4 by) % 16's value.
__device__ __forceinline__ u32x4 row_turn(const u32x4& v, int by) {
  u32x4 o = v;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    o[e] = by == 0   ? v[e]
           : by == 1 ? (uint32_t)__builtin_amdgcn_mov_dpp((int)v[e], 0x12C, 0xF, 0xF, true)   // row_ror:12
           : by == 2 ? (uint32_t)__builtin_amdgcn_mov_dpp((int)v[e], 0x128, 0xF, 0xF, true)   // row_ror:8
                     : (uint32_t)__builtin_amdgcn_mov_dpp((int)v[e], 0x124, 0xF, 0xF, true);  // row_ror:4
  return o;
}

// The scale fields of block blk = 4 q' + grp as loaded, and at their use. kWhole
// (K % 256 == 0, so that a row's blocks come in whole fours): as the 32-bit word
// that holds them, whose part is taken at the use. (A byte or half carried from
// one chunk to the next is widened, and so waited for, where the branch of a
// row group's end has come between: the ring drained every third chunk.)
template <int kForm, bool kWhole>
__device__ __forceinline__ void pair_scale_load(const i32x4& c8r, const i32x4& s2r, uint32_t blk, uint32_t& c8,
                                                uint32_t& s2) {
  if constexpr (kWhole) {
    c8 = kForm == 0 ? raw_buffer_load_u32(c8r, (int)(blk & ~3u), 0, 0) : 0u;
    s2 = raw_buffer_load_u32(s2r, (int)(kForm == 0 ? blk / kDqBlock * 4 : kForm == 1 ? blk * 4 : (blk & ~1u) * 2), 0, 0);
  } else {
    float v;
    scale_fields_of<kForm>(c8r, s2r, blk, c8, v);
    s2 = __builtin_bit_cast(uint32_t, v);
  }
}

template <int kForm, bool kWhole>
__device__ __forceinline__ float pair_scale(uint32_t c8, uint32_t s2, int grp, float mean) {
  if constexpr (kWhole) {
    c8 = kForm == 0 ? (c8 >> (8 * grp)) & 0xFFu : (uint32_t)kE4m3One;
    if constexpr (kForm == 2) s2 = (grp & 1) ? s2 & 0xFFFF0000u : s2 << 16;
  }
  return decode_block_scale(c8, __builtin_bit_cast(float, s2), mean);
}

// kX: see above; kForm: the block-scale form (scale_fields_of). G and U may be NULL; L NULL: no adapters.
template <int kX, bool kF16, int kForm, bool kWhole>
__global__ __launch_bounds__(64 * kPW) void gemv_pair_kernel(PairWeight wg, PairWeight wu, int64_t N, int64_t K,
                                                             const uint16_t* __restrict__ X,
                                                             const u32x4* __restrict__ Xp, int64_t M,
                                                             const float* __restrict__ L, uint16_t* __restrict__ H,
                                                             uint16_t* __restrict__ G, uint16_t* __restrict__ U) {
  // table entry b (a code byte): the levels of its two codes, 32 copies of 8
  // bytes, so that a lane's address is its code byte in bits 8..15 and its
  // copy's offset below (one byte permute). Where the two codebooks are equal
  // (the usual case) all are alike, else the first 16 are the gate's and the
  // others the up's.
  __shared__ __attribute__((aligned(16))) char lut[256 * 256];
  // (three ring arrays, so the compiler can tell the one being read from those being filled)
  __shared__ __attribute__((aligned(16))) char ring0[kPW * kSlot];
  __shared__ __attribute__((aligned(16))) char ring1[kPW * kSlot];
  __shared__ __attribute__((aligned(16))) char ring2[kPW * kSlot];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  // the levels pass through the first ring (not yet in use)
  float* const levels = reinterpret_cast<float*>(ring0);
  if (t < 16) {
    levels[t] = wg.codebook[t];
    levels[16 + t] = wu.codebook[t];
  }
  __syncthreads();
  const bool same = __ballot(__float_as_uint(levels[lane & 15]) != __float_as_uint(levels[16 + (lane & 15)])) == 0;
  for (int i = t; i < 256 * 32; i += 64 * kPW) {
    const int e = i >> 5;
    const float* const lv = same || (i & 31) < 16 ? levels : levels + 16;
    reinterpret_cast<float2*>(lut)[i] = float2{lv[e & 15], lv[e >> 4]};
  }
  const float mean[2] = {weight_mean(wg.code8, wg.mean), weight_mean(wu.code8, wu.mean)};
  const int nq = (int)cdiv(K, (int64_t)256);
  const int per = (nq + kPW - 1) / kPW;  // chunks per wave and row group: wave, wave + 8, ...
  const int tiles = (int)cdiv(N, (int64_t)16);
  const int items = (tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x * per;
  const int grp = lane >> 4;  // which 64-block of a chunk
  const int col = lane & 15;  // A: token; B: weight row within a tile
  const int64_t kblocks = K / kBlock;

  // Copies: lane l of copy h fills row 8 h + l / 8 of a tile at swizzled
  // position l % 8. Rows past N lie past the end of the codes and read as
  // zero; columns past K in the last chunk read the next row's codes and meet
  // zero activations.
  const i32x4 crs[2] = {make_rsrc(wg.codes, N * (K / 2)), make_rsrc(wu.codes, N * (K / 2))};
  uint32_t cvoff[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int rr = 8 * h + (lane >> 3);
    cvoff[h] = (uint32_t)(rr * (K / 2) + 16 * ((lane & 7) ^ code_swz(rr)));
  }
  const uint32_t rd0 = (uint32_t)(col * 128 + 16 * ((2 * grp) ^ code_swz(col)));
  const uint32_t off[2] = {(uint32_t)(same ? lane & 31 : lane & 15) * 8,
                           (uint32_t)(same ? lane & 31 : 16 + (lane & 15)) * 8};
  const i32x4 xrs = kX == kXOrder ? make_rsrc(Xp, (int64_t)nq * 512 * 16) : make_rsrc(X, M * K * 2);
  const uint32_t xvoff = kX == kXOrder  ? (uint32_t)lane * 16
                         : kX == kXFour ? (uint32_t)((col & 3) * K * 2 + 128 * grp + 16 * (col >> 2))
                                        : (uint32_t)(col * K * 2 + 128 * grp);
  const int64_t nblk = N * kblocks;
  const int64_t s2_bytes = kForm == 0 ? cdiv(nblk, (int64_t)kDqBlock) * 4 : nblk * (kForm == 1 ? 4 : 2);
  const i32x4 c8rs[2] = {make_rsrc(wg.code8, kForm == 0 ? nblk : 0), make_rsrc(wu.code8, kForm == 0 ? nblk : 0)};
  const i32x4 s2rs[2] = {make_rsrc(wg.s2, s2_bytes), make_rsrc(wu.s2, s2_bytes)};
  // wave w adds L of weight w % 2, token rows 4 g + w / 2, to its sums
  const i32x4 lrs = make_rsrc(L, L != nullptr ? 2 * M * N * 4 : 0);
  const int64_t lm = 4 * grp + (wave >> 1);
  const uint32_t lvoff = (uint32_t)((((wave & 1) * M + lm) * N + col) * 4);

  // the next chunk to be copied, and (below) the next to be worked on
  int ic = 0, left = items;
  uint32_t in0 = blockIdx.x * 16;
  auto issue = [&](char* R, PairStage<kX>& st) {
    const int q = wave + kPW * ic < nq ? wave + kPW * ic : nq - 1;  // (past the end: not worked on)
    char* const dst = R + wave * kSlot;
    const uint32_t row0 = in0 * (uint32_t)(K / 2);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) copy16(crs[i], row0 + cvoff[h], q * 128, dst + i * 2048 + h * 1024);
    const int kc = q * 256 + 64 * grp;
    const uint32_t n = in0 + col < N ? in0 + col : (uint32_t)(N - 1);
    const uint32_t blk = n * (uint32_t)kblocks + (uint32_t)(kWhole || kc < K ? kc / kBlock : kblocks - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) pair_scale_load<kForm, kWhole>(c8rs[i], s2rs[i], blk, st.c8[i], st.s2[i]);
    st.l = __builtin_bit_cast(
        float, raw_buffer_load_u32(lrs, (int)(lm < M && in0 + col < N ? lvoff + in0 * 4 : 0x80000000u), 0, 0));
    if constexpr (kX == kXOrder) {
#pragma unroll
      for (int s = 0; s < 8; ++s) st.xa[s] = raw_buffer_load_b128(xrs, (int)xvoff, q * 8192 + s * 1024, 0);
    } else {
      const uint32_t v = kWhole || kc < K ? xvoff : 0x80000000u;
#pragma unroll
      for (int s = 0; s < (kX == kXFour ? 2 : 8); ++s)
        st.xa[s] = raw_buffer_load_b128(xrs, (int)(v + (kX == kXFour ? 64 : 16) * s), q * 512, 0);
    }
    if (--left > 0 && ++ic == per) {  // (past the last: that one again)
      ic = 0;
      in0 += 16 * gridDim.x;
    }
  };

  f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
  // One chunk, one code word of each weight at a time: the table reads of word
  // s + 1 are issued before the products of word s, and the two products of a
  // word add to different sums.
  auto compute = [&](const char* R, const PairStage<kX>& st) {
    const char* const src = R + wave * kSlot;
    uint32_t cw[2][8];
    float cp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 c0 = *reinterpret_cast<const u32x4*>(src + i * 2048 + rd0);
      const u32x4 c1 = *reinterpret_cast<const u32x4*>(src + i * 2048 + (rd0 ^ 16u));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cw[i][e] = c0[e];
        cw[i][4 + e] = c1[e];
      }
      cp[i] = pair_scale<kForm, kWhole>(st.c8[i], st.s2[i], grp, mean[i]);
    }
    float2 lv[2][8];
    auto gather = [&](int s, float2 (&out)[8]) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int p = 0; p < 4; ++p)
          out[4 * i + p] = *reinterpret_cast<const float2*>(
              lut + __builtin_amdgcn_perm(cw[i][s], off[i], 0x0C0C0400u + ((uint32_t)p << 8)));
    };
    gather(0, lv[0]);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      // (one wait for all of word s's reads)
      if (s + 1 < 8) {
        gather(s + 1, lv[(s + 1) & 1]);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(lgkm_wait(8));
      } else {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(lgkm_wait(0));
      }
      __builtin_amdgcn_sched_barrier(0);
      u32x4 xa;
      if constexpr (kX == kXFour)
        xa = row_turn(st.xa[s >> 2], s & 3);
      else
        xa = st.xa[s];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        u32x4 bw;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float2 l = lv[s & 1][4 * i + p];
          bw[p] = pack2<kF16>(nf4_scaled(l.x, cp[i]), nf4_scaled(l.y, cp[i]));
        }
        acc[i] = mfma16<kF16>(__builtin_bit_cast(bf16x8, xa), __builtin_bit_cast(bf16x8, bw), acc[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // (a barrier that leaves the copies in flight)
  auto meet = [] {
    __builtin_amdgcn_s_waitcnt(lgkm_wait(0));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // One chunk, and after the last of every second row group (and of the very
  // last) the join of both: the waves' sums, each in its own slot of the ring
  // array just read (free until the next copies go there), are added in wave
  // order, 256 threads per row group. (28672 x 8192, one token: 63 us; a join
  // for every row group 66.)
  int cc = 0, groups = items / per;
  bool held = false;
  f32x4 hold[2] = {acc[0], acc[1]};
  int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t nstep = 16 * (int64_t)gridDim.x;
  auto step = [&](char* R, const PairStage<kX>& st) {
    if (wave + kPW * cc < nq) compute(R, st);
    if (++cc < per) return;
    cc = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][v] += wave == 2 * v + i ? st.l : 0.0f;
    if (--groups > 0 && !held) {
      held = true;
      hold[0] = acc[0];
      hold[1] = acc[1];
    } else {
      float(*mine)[2][16][16] = reinterpret_cast<float(*)[2][16][16]>(R + wave * kSlot);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          mine[0][i][4 * grp + v][col] = acc[i][v];
          mine[1][i][4 * grp + v][col] = hold[i][v];
        }
      meet();
      const int m = (t >> 4) & 15, nc = t & 15;
      const int64_t n = n0 + nc - (t >> 8) * nstep;  // the second half of the threads: the group before
      if (m < M && n < N && (held || t < 256)) {
        float y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float* const s = reinterpret_cast<const float*>(R) + (((t >> 8) * 2 + i) * 16 + m) * 16 + nc;
          y[i] = s[0];
#pragma unroll
          for (int w = 1; w < kPW; ++w) y[i] += s[w * (kSlot / 4)];
        }
        const int64_t o = m * N + n;
        H[o] = to16<kF16>(silu(y[0]) * y[1]);
        if (G) G[o] = to16<kF16>(y[0]);
        if (U) U[o] = to16<kF16>(y[1]);
      }
      meet();
      held = false;
    }
    acc[0] = acc[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    n0 += nstep;
  };

  __syncthreads();  // the table (and the levels read before the copies reuse the first ring)
  PairStage<kX> st0, st1, st2;
  issue(ring0, st0);
  issue(ring1, st1);
  // whole groups of three chunks, with no exit inside a group (a path on which
  // a chunk's loads are still pending at the loop's head makes the compiler
  // wait for every load there)
  int j = 0;
  for (; j + 3 <= items; j += 3) {
    issue(ring2, st2);
    __builtin_amdgcn_sched_barrier(0);
    step(ring0, st0);
    __builtin_amdgcn_sched_barrier(0);
    issue(ring0, st0);
    __builtin_amdgcn_sched_barrier(0);
    step(ring1, st1);
    __builtin_amdgcn_sched_barrier(0);
    issue(ring1, st1);
    __builtin_amdgcn_sched_barrier(0);
    step(ring2, st2);
    __builtin_amdgcn_sched_barrier(0);
  }
  if (j < items) step(ring0, st0);
  if (j + 1 < items) step(ring1, st1);
  // (copies past the range may still be landing: done before the workgroup's LDS is another's)
  __builtin_amdgcn_s_waitcnt(0);
}

// Column ranges of the projections: about one 128-column block per wave, at
// most 16 workgroups.
struct PairPlan {
  int nb, chunk, parts;
};

PairPlan pair_plan(int64_t k) {
  const int nb = (int)(2 * cdiv(k, (int64_t)256));
  const int chunk = cdiv(nb, 16) > 4 ? (int)cdiv(nb, 16) : 4;
  return PairPlan{nb, chunk, (int)cdiv(nb, chunk)};
}

}  // namespace

size_t gemv_pair_ws_bytes(int64_t M, int64_t n, int64_t k, int r) {
  return gemv_ws_bytes(k) + align256((size_t)pair_plan(k).parts * 2 * M * r * 4) + align256((size_t)(r > 0 ? 2 * M * n * 4 : 0));
}

hipError_t launch_gemv_pair(const Nf4View& g, const Nf4View& u, const uint16_t* X, int64_t M, const uint16_t* Ag,
                            const uint16_t* Bg, const uint16_t* Au, const uint16_t* Bu, int r, float scale, uint16_t* H,
                            uint16_t* G, uint16_t* U, float* T_save, void* ws, hipStream_t stream, bool f16) {
  if (!gemv_fits(g.n, g.k) || M > 16) return hipErrorInvalidValue;
  u32x4* const Xp = static_cast<u32x4*>(ws);
  const PairPlan pl = pair_plan(g.k);
  float* const part = reinterpret_cast<float*>(static_cast<char*>(ws) + gemv_ws_bytes(g.k));
  float* const L = r > 0 ? part + align256((size_t)pl.parts * 2 * M * r * 4) / 4 : nullptr;
  const bool xp = M > 4 && gemv_orders_x(M, g.n);
  if (xp || r > 0) {
#define QLORA_GPREP2(RP, H16) \
  gemv_prep_kernel<RP, H16><<<(unsigned)pl.parts, 256, 0, stream>>>(X, M, g.k, pl.nb, Ag, Au, r, pl.chunk, xp ? Xp : nullptr, part)
#define QLORA_GPREP(RP) { if (f16) QLORA_GPREP2(RP, true); else QLORA_GPREP2(RP, false); }
    if (r == 0) QLORA_GPREP(0)
    else if (r <= 16) QLORA_GPREP(16)
    else if (r <= 32) QLORA_GPREP(32)
    else if (r <= 64) QLORA_GPREP(64)
    else QLORA_GPREP(128)
#undef QLORA_GPREP
#undef QLORA_GPREP2
  }
  if (r > 0) {
    const unsigned grid = (unsigned)cdiv(g.n, (int64_t)64);
    if (f16)
      pair_lowrank_kernel<true><<<grid, 256, 0, stream>>>(part, pl.parts, M, r, scale, Bg, Bu, g.n, T_save, L);
    else
      pair_lowrank_kernel<false><<<grid, 256, 0, stream>>>(part, pl.parts, M, r, scale, Bg, Bu, g.n, T_save, L);
  }
  const PairWeight wg{g.codes, g.code8, g.s2, g.mean, g.codebook}, wu{u.codes, u.code8, u.s2, u.mean, u.codebook};
  const int64_t tiles = cdiv(g.n, (int64_t)16);
  const unsigned grid = (unsigned)(tiles < kPairGroups ? tiles : kPairGroups);
  const int form = g.code8 ? 0 : (g.s2_bf16 ? 2 : 1);
  const bool whole = g.k % 256 == 0;
#define QLORA_GVP4(XP, H16, F, W) \
  gemv_pair_kernel<XP, H16, F, W><<<grid, 64 * kPW, 0, stream>>>(wg, wu, g.n, g.k, X, Xp, M, L, H, G, U)
#define QLORA_GVP3(XP, H16, F) { if (whole) QLORA_GVP4(XP, H16, F, true); else QLORA_GVP4(XP, H16, F, false); }
#define QLORA_GVP2(XP, H16)                  \
  {                                          \
    if (form == 0) QLORA_GVP3(XP, H16, 0)    \
    else if (form == 1) QLORA_GVP3(XP, H16, 1) \
    else QLORA_GVP3(XP, H16, 2)              \
  }
#define QLORA_GVP(XP) { if (f16) QLORA_GVP2(XP, true) else QLORA_GVP2(XP, false) }
  if (M <= 4) QLORA_GVP(kXFour)
  else if (xp) QLORA_GVP(kXOrder)
  else QLORA_GVP(kXPlace)
#undef QLORA_GVP
#undef QLORA_GVP2
#undef QLORA_GVP3
#undef QLORA_GVP4
  return hipGetLastError();
}

}  // namespace qlora
