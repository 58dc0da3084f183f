// The gradient through a matrix product's epilogue (declared in include/nvfp4.h): elementwise, with
// the bias's gradient (column sums) and the amax of what it writes from the same pass. Bound by DRAM:
// two reads and a write of 2 bytes an element.
//
// A CTA of 256 threads has 2048 columns, a thread eight of them, over a range of rows; its column sums
// go to one row of the partial sums, which a second kernel adds up in order.
#include <cuda_bf16.h>
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

constexpr int kThreads = 256;

template <int ACT>
__global__ void __launch_bounds__(kThreads) epilogue_backward_kernel(
    const uint4* grad, const uint4* z, int64_t M, int64_t nv, uint4* out, float* partial, int64_t rows,
    uint32_t* amax) {
  pdl_wait();
  pdl_allow_next();
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t first = (int64_t)blockIdx.y * rows, last = min(first + rows, M);
  float sum[8] = {};
  uint32_t top = 0u;
  if (c < nv) {
    for (int64_t r = first; r < last; r++) {
      const uint4 gv = grad[r * nv + c], zv = z[r * nv + c];
      const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w}, zw[4] = {zv.x, zv.y, zv.z, zv.w};
      uint32_t ow[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        float d[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const float g = __uint_as_float(h ? gw[j] & 0xFFFF0000u : gw[j] << 16);
          const float x = __uint_as_float(h ? zw[j] & 0xFFFF0000u : zw[j] << 16);
          d[h] = g * activation_slope<ACT>(x);
          sum[2 * j + h] += d[h];
        }
        const __nv_bfloat162 p = __floats2bfloat162_rn(d[0], d[1]);
        ow[j] = *reinterpret_cast<const uint32_t*>(&p);
        top = max(top, max(ow[j] & 0x7FFFu, (ow[j] >> 16) & 0x7FFFu));
      }
      out[r * nv + c] = make_uint4(ow[0], ow[1], ow[2], ow[3]);
    }
    if (partial != nullptr) {
      float4* const to = reinterpret_cast<float4*>(partial) + ((int64_t)blockIdx.y * nv + c) * 2;
      to[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
      to[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
    }
  }
  if (amax != nullptr) {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0 && m != 0u) atomicMax(amax, m << 16);
  }
}

__global__ void __launch_bounds__(kThreads) column_sum_kernel(const float* partial, int64_t rows, int64_t N,
                                                              float* out) {
  pdl_wait();
  pdl_allow_next();
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= N) return;
  float s = 0.0f;
  for (int64_t r = 0; r < rows; r++) s += partial[r * N + c];
  out[c] = s;
}

}  // namespace

cudaError_t launch_epilogue_backward(const void* grad, const void* preact, int64_t M, int64_t N,
                                     int32_t activation, void* grad_z, float* grad_bias, float* amax,
                                     float* partial, int sm_count, cudaStream_t s) {
  const int64_t nv = N / 8, across = (nv + kThreads - 1) / kThreads;
  // ranges of rows: about four CTAs an SM in all, at most the rows of the workspace
  int64_t down = (4 * sm_count + across - 1) / across;
  if (down > kEpilogueMaxPartials) down = kEpilogueMaxPartials;
  if (down > M) down = M;
  const int64_t rows = (M + down - 1) / down;
  down = (M + rows - 1) / rows;
  const dim3 grid((unsigned)across, (unsigned)down), block(kThreads);
  auto run = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, s, static_cast<const uint4*>(grad),
                      static_cast<const uint4*>(preact), M, nv, static_cast<uint4*>(grad_z),
                      grad_bias ? partial : nullptr, rows, reinterpret_cast<uint32_t*>(amax));
  };
  cudaError_t e;
  switch (activation) {
    case NVFP4_ACT_RELU: e = run(epilogue_backward_kernel<NVFP4_ACT_RELU>); break;
    case NVFP4_ACT_RELU2: e = run(epilogue_backward_kernel<NVFP4_ACT_RELU2>); break;
    case NVFP4_ACT_GELU: e = run(epilogue_backward_kernel<NVFP4_ACT_GELU>); break;
    case NVFP4_ACT_SILU: e = run(epilogue_backward_kernel<NVFP4_ACT_SILU>); break;
    default: e = run(epilogue_backward_kernel<NVFP4_ACT_NONE>);
  }
  if (e != cudaSuccess || grad_bias == nullptr) return e;
  return launch_pdl(column_sum_kernel, dim3((unsigned)((N + kThreads - 1) / kThreads)), block, 0, s,
                    (const float*)partial, down, N, grad_bias);
}

}  // namespace nvfp4
