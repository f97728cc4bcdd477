// Host-side helpers shared by the C ABI's entry points.
#pragma once

#include <cstdint>

#include "kernels.h"
#include "qlora.h"

namespace qlora {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A buffer that a call reads or writes: present and 16-byte aligned.
inline bool good(const void* p) { return p != nullptr && aligned16(p); }

inline qlora_status hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP; }

// Largest M, n and k of the feed-forward calls: keeps every element count
// and grid within 64- and 32-bit arithmetic.
constexpr int64_t kMaxDim = (int64_t)1 << 22;

qlora_status check_weight(const qlora_nf4_weight* w);
Nf4View view_of(const qlora_nf4_weight* w);

// Zeros for the adapter gradients of an empty batch (a kernel, not a memset,
// so the call stays capturable in a graph).
hipError_t zero_f32(float* p, int64_t n, hipStream_t st);

// Bump allocator over the caller's workspace (256-byte aligned regions).
struct Carver {
  char* base;
  size_t used = 0;
  explicit Carver(void* p) : base(static_cast<char*>(p)) {}
  template <typename T>
  T* take(size_t bytes) {
    if (bytes == 0) return nullptr;
    T* p = reinterpret_cast<T*>(base ? base + used : nullptr);
    used += align256(bytes);
    return p;
  }
};

}  // namespace qlora
