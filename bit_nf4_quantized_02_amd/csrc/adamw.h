// The AdamW update of one element, shared by the step over one tensor and the
// step over many.
#pragma once

#include "common.h"
#include "qlora.h"

namespace qlora {

struct AdamwC {
  float b1, b2, omb1, omb2, lr, eps, wd, bc1, bc2;
};

__device__ __forceinline__ void adamw_one(float& th, float g, float& m, float& v, const AdamwC& c) {
#pragma clang fp contract(off)
  m = c.b1 * m + c.omb1 * g;
  v = c.b2 * v + c.omb2 * (g * g);
  const float mhat = m / c.bc1;
  const float vhat = v / c.bc2;
  const float u = mhat / (sqrtf(vhat) + c.eps) + c.wd * th;
  th = th - c.lr * u;
}

// The step's constants (1 - b1, 1 - b2 and the bias corrections formed in fp64
// and rounded once); false for hyperparameters out of range.
bool adamw_constants(int64_t step, float lr, float beta1, float beta2, float eps, float weight_decay, AdamwC& c);

// Device address of an optimizer state: device memory as is, pinned host memory
// through its device mapping; false for anything else (pageable host memory,
// unknown pointers).
bool state_ptr(float* p, float** dev);

}  // namespace qlora
