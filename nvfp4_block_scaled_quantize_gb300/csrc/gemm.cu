// Matrix products of NVFP4 operands (declared in include/nvfp4.h).
//
// First form: a CTA has a 64 x 64 tile of out, its operands' 16-element blocks decoded to binary32 in
// shared memory, a thread 4 x 4 sums.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4.h"
#include "nvfp4_device.cuh"
#include "aux_internal.h"
#include "gemm_device.cuh"
#include "gemm_internal.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, f = c & 1u;
  const float v = e == 0 ? 0.5f * f : (1.0f + 0.5f * f) * (float)(1 << (e - 1));
  return (c & 8u) ? -v : v;
}
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half2float(__ushort_as_half((unsigned short)h));
}
__device__ __forceinline__ float act_any(int act, float z) {
  switch (act) {
    case NVFP4_ACT_RELU: return activate<NVFP4_ACT_RELU>(z);
    case NVFP4_ACT_RELU2: return activate<NVFP4_ACT_RELU2>(z);
    case NVFP4_ACT_GELU: return activate<NVFP4_ACT_GELU>(z);
    case NVFP4_ACT_SILU: return activate<NVFP4_ACT_SILU>(z);
  }
  return z;
}

__global__ void __launch_bounds__(256) gemm_simple_kernel(const GemmArgs g) {
  __shared__ float sa[16][65], sb[16][65];
  pdl_wait();
  pdl_allow_next();
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  int e = blockIdx.z;
  int64_t row0 = 0, rows = g.M, k0 = 0, k1 = g.K, batch = 0, out0 = 0;
  if (g.mode == kGemmGrouped) {
    row0 = e == 0 ? 0 : g.offsets[e - 1];
    const int64_t end = g.offsets[e];
    if (row0 < 0 || end < row0 || end > g.M) {
      if (threadIdx.x == 0) atomicOr(g.status, 1u);
      return;
    }
    rows = end - row0;
    batch = e;
  } else if (g.mode == kGemmWgrad) {
    int64_t prev = 0, at = 0;
    for (int i = 0; i <= e; i++) {
      const int64_t end = g.offsets[i];
      if (end < prev) {
        if (threadIdx.x == 0) atomicOr(g.status, 1u);
        return;
      }
      k0 = at;
      at += (end - prev + 15) / 16 * 16;
      prev = end;
    }
    k1 = at;
    if (k1 > g.K) {
      if (threadIdx.x == 0) atomicOr(g.status, 1u);
      return;
    }
    out0 = (int64_t)e * g.M * g.N;
  } else {
    e = 0;
  }
  const float alpha = g.a.gscale[2 * e + 1] * g.b.gscale[2 * e + 1];
  float top = 0.0f;
  const int64_t n0 = (int64_t)blockIdx.y * 64;
  for (int64_t m0 = (int64_t)blockIdx.x * 64; m0 < rows; m0 += (int64_t)gridDim.x * 64) {
    float acc[4][4] = {};
    for (int64_t k = k0; k < k1; k += 16) {
      for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int r = i / 8, c = i % 8;
        const int64_t m = row0 + m0 + r, n = n0 + r;
        float v = 0.0f, w = 0.0f, v2 = 0.0f, w2 = 0.0f;
        if (m0 + r < rows) {
          const uint32_t b = g.a.codes[m * g.a.code_pitch + k / 2 + c];
          const float s = e4m3_value(g.a.scales[m * g.a.scale_pitch + k / 16]);
          v = e2m1_value(b & 15) * s, v2 = e2m1_value(b >> 4) * s;
        }
        if (n < g.N) {
          const uint32_t b = g.b.codes[batch * g.b.code_batch + n * g.b.code_pitch + k / 2 + c];
          const float s = e4m3_value(g.b.scales[batch * g.b.scale_batch + n * g.b.scale_pitch + k / 16]);
          w = e2m1_value(b & 15) * s, w2 = e2m1_value(b >> 4) * s;
        }
        sa[2 * c][r] = v, sa[2 * c + 1][r] = v2;
        sb[2 * c][r] = w, sb[2 * c + 1][r] = w2;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 16; c++)
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int j = 0; j < 4; j++)
            acc[i][j] = __fmaf_rn(sa[c][ty + 16 * i], sb[c][tx + 16 * j], acc[i][j]);
      __syncthreads();
    }
    for (int i = 0; i < 4; i++)
      for (int j = 0; j < 4; j++) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m >= rows || n >= g.N) continue;
        float z = acc[i][j] * alpha;
        const int64_t bn = (int64_t)e * g.N + n;
        if (g.bias)
          z += g.bias_bytes == 4 ? static_cast<const float*>(g.bias)[bn]
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(g.bias)[bn]);
        const int64_t at = out0 + (row0 + m) * g.N + n;
        if (g.preact) static_cast<__nv_bfloat16*>(g.preact)[at] = __float2bfloat16_rn(z);
        float o = act_any(g.activation, z);
        if (g.out_bytes == 4) {
          if (g.residual) o += static_cast<const float*>(g.residual)[at];
          static_cast<float*>(g.out)[at] = o;
        } else {
          if (g.residual) o += __bfloat162float(static_cast<const __nv_bfloat16*>(g.residual)[at]);
          const __nv_bfloat16 b = __float2bfloat16_rn(o);
          static_cast<__nv_bfloat16*>(g.out)[at] = b;
          o = __bfloat162float(b);
        }
        top = fmaxf(top, fabsf(o));
      }
  }
  if (g.amax) atomicMax(reinterpret_cast<uint32_t*>(g.amax) + e, __float_as_uint(top));
  if (g.mode == kGemmGrouped && e == g.E - 1) {
    const int64_t end = g.offsets[e];
    for (int64_t m = end + blockIdx.x; m < g.M; m += gridDim.x)
      for (int64_t n = n0 + threadIdx.x; n < g.N && n < n0 + 64; n += 256) {
        if (g.out_bytes == 4) static_cast<float*>(g.out)[m * g.N + n] = 0.0f;
        else static_cast<uint16_t*>(g.out)[m * g.N + n] = 0;
        if (g.preact) static_cast<uint16_t*>(g.preact)[m * g.N + n] = 0;
      }
  }
}

}  // namespace

cudaError_t prepare_gemm_kernels() { return cudaSuccess; }

cudaError_t launch_gemm(const GemmArgs& g, int sm_count, cudaStream_t s) {
  const int64_t mt = (g.M + 63) / 64;
  const dim3 grid((unsigned)(g.mode == kGemmGrouped ? (mt < 64 ? mt : 64) : mt),
                  (unsigned)((g.N + 63) / 64), g.mode == kGemmDense ? 1 : g.E);
  return launch_pdl(gemm_simple_kernel, grid, dim3(256), 0, s, g);
}

}  // namespace nvfp4
