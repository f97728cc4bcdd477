// What a training step does to all adapters' tensors together: the norm of
// their gradients, and the AdamW step scaled to a largest norm.
//
//   norm = s sqrt(sum g^2) over every element of every tensor (s: grad_scale)
//   factor = max_norm / norm if norm > max_norm, else 1 (NaN: a gradient is not finite)
//   AdamW (adamw.h) on s factor g
//
// The tensors are cut into chunks once, each described by a record of its own
// (addresses, length, types), so that one launch covers hundreds of tensors of
// any sizes and a workgroup finds its work with one scalar load. The factor
// stays on the device: neither the host nor a pass that rewrites the gradients
// stands between the norm and the step.
//
// Both are bound by HBM (a gradient is read once for each; theta, m and v are
// read and written once). Squares are added in fp64: no gradient of any
// magnitude overflows or vanishes, and the order (chunks of a workgroup, lanes,
// workgroups) is fixed. Measured (160 M fp32 gradients in 448 tensors): norm 104 us
// (6.1 TB/s), step 770 - 800 (5.3 TB/s), both 905.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "adamw.h"
#include "api_util.h"

namespace qlora {
namespace {

struct Chunk {
  float *theta, *m, *v;
  const void* grad;
  uint16_t* theta16;
  uint32_t count;
  uint32_t kinds;  // bits 0, 1: the gradient's qlora_dtype; bit 2: theta16 is fp16
};
static_assert(sizeof(Chunk) == 48, "the image's layout");

// Elements of a chunk: four for each thread of a workgroup, which then has all of
// its loads in flight at once and nothing to wait for before it ends (160 M
// parameters, step: 794 us; 2048 elements in a loop 859, 4096 877, 16384 921).
// A multiple of 64: every chunk starts as aligned as its tensor.
constexpr int kThreads = 256, kChunk = 4 * kThreads;
constexpr int64_t kMostChunks = (int64_t)1 << 23;  // (a launch has less than 2^32 threads)
constexpr int kMostGroups = 2048;  // workgroups of the norm, and its partial sums
constexpr int kTogether = 4;       // chunks that a workgroup of the norm reads at once

// Four consecutive gradients from element i on, in fp32; kind: qlora_dtype.
__device__ __forceinline__ float4 grad4(const void* g, int kind, int64_t i) {
  if (kind == QLORA_DT_FP32) return *reinterpret_cast<const float4*>(static_cast<const float*>(g) + i);
  const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(g) + i);
  if (kind == QLORA_DT_FP16)
    return float4{from16<true>(v[0] & 0xFFFFu), from16<true>(v[0] >> 16), from16<true>(v[1] & 0xFFFFu), from16<true>(v[1] >> 16)};
  return float4{from16<false>(v[0] & 0xFFFFu), from16<false>(v[0] >> 16), from16<false>(v[1] & 0xFFFFu), from16<false>(v[1] >> 16)};
}

__device__ __forceinline__ float grad1(const void* g, int kind, int64_t i) {
  if (kind == QLORA_DT_FP32) return static_cast<const float*>(g)[i];
  const uint16_t b = static_cast<const uint16_t*>(g)[i];
  return kind == QLORA_DT_FP16 ? from16<true>(b) : from16<false>(b);
}

__device__ __forceinline__ double square(float x, double s) { return fma((double)x, (double)x, s); }

// Sum over the workgroup in a fixed order, in thread 0. red: one for each wave.
template <int kWaves>
__device__ __forceinline__ double group_sum(double s, double* red) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  s = red[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) s += red[i];
  return s;
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const Chunk* __restrict__ chunks, int64_t n,
                                                             double* __restrict__ part) {
  __shared__ double red[kThreads / 64];
  const int t = threadIdx.x;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  for (int64_t b = (int64_t)blockIdx.x * kTogether; b < n; b += (int64_t)gridDim.x * kTogether) {
    float4 g[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const Chunk& c = chunks[b + j < n ? b + j : n - 1];
      const int kind = c.kinds & 3, count = b + j < n ? (int)c.count : 0;
      g[j] = float4{0.0f, 0.0f, 0.0f, 0.0f};
      if (4 * t + 4 <= count) {
        g[j] = grad4(c.grad, kind, 4 * t);
      } else {  // the end of a tensor
        if (4 * t < count) g[j].x = grad1(c.grad, kind, 4 * t);
        if (4 * t + 1 < count) g[j].y = grad1(c.grad, kind, 4 * t + 1);
        if (4 * t + 2 < count) g[j].z = grad1(c.grad, kind, 4 * t + 2);
      }
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      s[0] = square(g[j].x, s[0]);
      s[1] = square(g[j].y, s[1]);
      s[2] = square(g[j].z, s[2]);
      s[3] = square(g[j].w, s[3]);
    }
  }
  const double all = group_sum<kThreads / 64>((s[0] + s[1]) + (s[2] + s[3]), red);
  if (t == 0) part[blockIdx.x] = all;
}

__global__ __launch_bounds__(1024) void grad_factor_kernel(const double* __restrict__ part, int n, double scale,
                                                           double max_norm, float* __restrict__ out) {
  __shared__ double red[16];
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kMostGroups / 1024; ++i) {
    const int p = i * 1024 + (int)threadIdx.x;
    s += p < n ? part[p] : 0.0;
  }
  s = group_sum<16>(s, red);
  if (threadIdx.x != 0) return;
  const double norm = scale * sqrt(s);
  out[0] = (float)norm;
  out[1] = !isfinite(s) ? __uint_as_float(0x7FC00000u) : norm > max_norm ? (float)(max_norm / norm) : 1.0f;
}

// A chunk per workgroup, the last one first: the end of the gradients is what
// the norm's pass has left in the last-level cache, and theta, m and v, which are
// not used again, are read and written past it (nontemporal).
__global__ __launch_bounds__(kThreads) void adamw_many_kernel(const Chunk* __restrict__ chunks, int64_t n,
                                                              const float* __restrict__ clip, float scale, AdamwC k) {
  const Chunk c = chunks[n - 1 - blockIdx.x];
  float gs = scale;
  if (clip != nullptr) {
    const float factor = clip[1];
    if (isnan(factor)) return;  // a gradient is not finite: no step
    gs = scale * factor;
  }
  const int kind = c.kinds & 3, i = 4 * (int)threadIdx.x;
  const bool f16 = (c.kinds & 4) != 0;
  if (i + 4 <= (int)c.count) {
    f32x4* const tp = reinterpret_cast<f32x4*>(c.theta + i);
    f32x4* const mp = reinterpret_cast<f32x4*>(c.m + i);
    f32x4* const vp = reinterpret_cast<f32x4*>(c.v + i);
    const float4 g = grad4(c.grad, kind, i);
    const f32x4 t4 = __builtin_nontemporal_load(tp), m4 = __builtin_nontemporal_load(mp),
                v4 = __builtin_nontemporal_load(vp);
    const float gx[4] = {g.x * gs, g.y * gs, g.z * gs, g.w * gs};
    float th[4], m[4], v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      th[e] = t4[e];
      m[e] = m4[e];
      v[e] = v4[e];
      adamw_one(th[e], gx[e], m[e], v[e], k);
    }
    __builtin_nontemporal_store(f32x4{th[0], th[1], th[2], th[3]}, tp);
    __builtin_nontemporal_store(f32x4{m[0], m[1], m[2], m[3]}, mp);
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, vp);
    if (c.theta16 != nullptr)
      *reinterpret_cast<u32x2*>(c.theta16 + i) = f16 ? u32x2{pack2<true>(th[0], th[1]), pack2<true>(th[2], th[3])}
                                                     : u32x2{pack2<false>(th[0], th[1]), pack2<false>(th[2], th[3])};
    return;
  }
#pragma unroll 1
  for (int e = i; e < (int)c.count; ++e) {  // the end of a tensor
    float th = c.theta[e], m = c.m[e], v = c.v[e];
    adamw_one(th, grad1(c.grad, kind, e) * gs, m, v, k);
    c.theta[e] = th;
    c.m[e] = m;
    c.v[e] = v;
    if (c.theta16 != nullptr) c.theta16[e] = f16 ? to16<true>(th) : to16<false>(th);
  }
}

// The tensors' sizes and types, and how many elements and chunks they have.
qlora_status survey(const qlora_param* p, int64_t n, int64_t& elements, int64_t& chunks) {
  if (n < 0 || n > kMaxDim) return QLORA_ERR_SHAPE;
  if (p == nullptr && n > 0) return QLORA_ERR_INVALID_ARG;
  elements = chunks = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (p[i].count < 0 || p[i].count > ((int64_t)1 << 40)) return QLORA_ERR_SHAPE;
    elements += p[i].count;
    chunks += cdiv(p[i].count, (int64_t)kChunk);
  }
  return chunks > kMostChunks ? QLORA_ERR_SHAPE : QLORA_OK;
}

int grad_bytes(int dtype) { return dtype == QLORA_DT_FP32 ? 4 : 2; }

// Bytes that a tensor occupies, and whether the step writes them.
struct Span {
  uintptr_t from, to;
  bool written;
};

// No byte that the step writes belongs to anything else (two chunks would race).
bool apart(std::vector<Span>& s) {
  std::sort(s.begin(), s.end(), [](const Span& a, const Span& b) { return a.from < b.from; });
  uintptr_t any = 0, written = 0;
  for (const Span& x : s) {
    if (x.from < written || (x.written && x.from < any)) return false;
    any = std::max(any, x.to);
    if (x.written) written = std::max(written, x.to);
  }
  return true;
}

bool table_ok(const qlora_param_table* t) {
  return t != nullptr && t->n_chunks >= 0 && t->n_chunks <= kMostChunks && (t->n_chunks == 0 || good(t->chunks));
}

}  // namespace
}  // namespace qlora

using namespace qlora;

extern "C" {

size_t qlora_param_table_bytes(const qlora_param* params, int64_t n) {
  int64_t elements, chunks;
  return survey(params, n, elements, chunks) == QLORA_OK ? (size_t)chunks * sizeof(Chunk) : 0;
}

qlora_status qlora_param_table_build(const qlora_param* params, int64_t n, void* image, size_t image_bytes,
                                     qlora_param_table* table) {
  if (table == nullptr) return QLORA_ERR_INVALID_ARG;
  int64_t elements, chunks;
  const qlora_status s = survey(params, n, elements, chunks);
  if (s != QLORA_OK) return s;
  if (chunks > 0 && (image == nullptr || image_bytes < (size_t)chunks * sizeof(Chunk))) return QLORA_ERR_WORKSPACE;
  Chunk* out = static_cast<Chunk*>(image);
  bool complete = true;
  try {
    std::vector<Span> spans;
    for (int64_t i = 0; i < n; ++i) {
      const qlora_param& p = params[i];
      if (p.count == 0) continue;
      if (p.grad_dtype != QLORA_DT_FP32 && p.grad_dtype != QLORA_DT_BF16 && p.grad_dtype != QLORA_DT_FP16)
        return QLORA_ERR_INVALID_ARG;
      if (p.dtype16 != QLORA_DT_BF16 && p.dtype16 != QLORA_DT_FP16) return QLORA_ERR_INVALID_ARG;
      if (!good(p.grad)) return QLORA_ERR_INVALID_ARG;
      const bool whole = p.theta != nullptr;
      float *m = nullptr, *v = nullptr;
      if (whole) {
        if (!good(p.theta) || !good(p.m) || !good(p.v) || !aligned16(p.theta16)) return QLORA_ERR_INVALID_ARG;
        if (!state_ptr(p.m, &m) || !state_ptr(p.v, &v) || !aligned16(m) || !aligned16(v)) return QLORA_ERR_INVALID_ARG;
      } else if (p.m != nullptr || p.v != nullptr || p.theta16 != nullptr) {
        return QLORA_ERR_INVALID_ARG;
      }
      complete = complete && whole;
      const auto span = [&](const void* a, int64_t bytes, bool w) {
        const uintptr_t f = reinterpret_cast<uintptr_t>(a);
        spans.push_back(Span{f, f + (uintptr_t)(p.count * bytes), w});
      };
      span(p.grad, grad_bytes(p.grad_dtype), false);
      if (whole) {
        span(p.theta, 4, true);
        span(m, 4, true);
        span(v, 4, true);
        if (p.theta16 != nullptr) span(p.theta16, 2, true);
      }
      for (int64_t at = 0; at < p.count; at += kChunk)
        *out++ = Chunk{whole ? p.theta + at : nullptr,
                       whole ? m + at : nullptr,
                       whole ? v + at : nullptr,
                       static_cast<const char*>(p.grad) + at * grad_bytes(p.grad_dtype),
                       p.theta16 != nullptr ? p.theta16 + at : nullptr,
                       (uint32_t)std::min<int64_t>(kChunk, p.count - at),
                       (uint32_t)p.grad_dtype | (p.dtype16 == QLORA_DT_FP16 ? 4u : 0u)};
    }
    if (!apart(spans)) return QLORA_ERR_INVALID_ARG;
  } catch (const std::bad_alloc&) {
    return QLORA_ERR_UNSUPPORTED;
  }
  table->n_chunks = chunks;
  table->elements = elements;
  table->complete = complete ? 1 : 0;
  return QLORA_OK;
}

size_t qlora_grad_norm_workspace_bytes(void) { return kMostGroups * sizeof(double); }

qlora_status qlora_grad_norm(const qlora_param_table* table, float grad_scale, float max_norm, float* out, void* ws,
                             size_t ws_bytes, void* stream) {
  if (!table_ok(table) || !good(out)) return QLORA_ERR_INVALID_ARG;
  if (!(grad_scale > 0.0f) || std::isinf(grad_scale) || !(max_norm > 0.0f)) return QLORA_ERR_INVALID_ARG;
  if (!good(ws) || ws_bytes < qlora_grad_norm_workspace_bytes()) return QLORA_ERR_WORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  double* const part = static_cast<double*>(ws);
  const int groups = (int)std::min<int64_t>(cdiv(table->n_chunks, (int64_t)kTogether), kMostGroups);
  if (groups > 0) grad_norm_kernel<<<groups, kThreads, 0, st>>>(static_cast<const Chunk*>(table->chunks), table->n_chunks, part);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) {
    grad_factor_kernel<<<1, 1024, 0, st>>>(part, groups, (double)grad_scale, (double)max_norm, out);
    e = hipGetLastError();
  }
  return hip_status(e);
}

qlora_status qlora_adamw_step_many(const qlora_param_table* table, const float* clip, float grad_scale, int64_t step,
                                   float lr, float beta1, float beta2, float eps, float weight_decay, void* stream) {
  if (!table_ok(table) || table->complete != 1) return QLORA_ERR_INVALID_ARG;
  if (step < 1) return QLORA_ERR_SHAPE;
  if (!aligned16(clip) || !(grad_scale > 0.0f) || std::isinf(grad_scale)) return QLORA_ERR_INVALID_ARG;
  AdamwC c;
  if (!adamw_constants(step, lr, beta1, beta2, eps, weight_decay, c)) return QLORA_ERR_INVALID_ARG;
  if (table->n_chunks == 0) return QLORA_OK;
  adamw_many_kernel<<<(unsigned)table->n_chunks, kThreads, 0, static_cast<hipStream_t>(stream)>>>(
      static_cast<const Chunk*>(table->chunks), table->n_chunks, clip, grad_scale, c);
  return hip_status(hipGetLastError());
}

}  // extern "C"
