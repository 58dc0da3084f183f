// Device functions shared by the matrix products and the gradient of their epilogue.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "nvfp4.h"

namespace nvfp4 {

// Activations in binary32. The tanh form of GELU is z * sigmoid(2 u), u = sqrt(2 / pi) (z + 0.044715
// z^3), since (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)): relative to the result it stays exact far from
// zero, where 1 + tanh cancels.
constexpr float kGeluC = 0.7978845608028654f, kGeluA = 0.044715f;

// 1 / (1 + exp(-x))
__device__ __forceinline__ float sigmoid(float x) {
  return __fdividef(1.0f, 1.0f + __expf(-x));
}
template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == NVFP4_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays
  if constexpr (ACT == NVFP4_ACT_RELU2) {
    const float r = z < 0.0f ? 0.0f : z;
    return r * r;
  }
  if constexpr (ACT == NVFP4_ACT_GELU)
    return z * sigmoid(2.0f * kGeluC * z * __fmaf_rn(kGeluA * z, z, 1.0f));
  if constexpr (ACT == NVFP4_ACT_SILU) return z * sigmoid(z);
  return z;
}
template <int ACT>
__device__ __forceinline__ float activation_slope(float z) {
  if constexpr (ACT == NVFP4_ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  if constexpr (ACT == NVFP4_ACT_RELU2) return z < 0.0f ? 0.0f : 2.0f * z;
  if constexpr (ACT == NVFP4_ACT_GELU) {
    // p = sigmoid(2u): p + z p (1 - p) 2 u'
    const float q = kGeluA * z * z;
    const float p = sigmoid(2.0f * kGeluC * z * (1.0f + q));
    const float du = 2.0f * kGeluC * (1.0f + 3.0f * q);
    return p * (1.0f + z * (1.0f - p) * du);
  }
  if constexpr (ACT == NVFP4_ACT_SILU) {
    const float p = sigmoid(z);
    return p * (1.0f + z * (1.0f - p));
  }
  return 1.0f;
}

}  // namespace nvfp4
