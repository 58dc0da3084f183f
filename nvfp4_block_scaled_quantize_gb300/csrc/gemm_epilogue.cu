// The gradient through a matrix product's epilogue (declared in include/nvfp4.h): elementwise, with
// the bias's gradient (column sums) and the amax of what it writes from the same pass. Bound by DRAM:
// two reads and a write of 2 bytes an element.
//
// A CTA of 128 threads has 2048 columns (1024 where rows do not start on 32-byte boundaries), a thread
// 16 (8) of them, over a range of rows, two at a time so that their loads are under way together. Its
// column sums go to one row of the partial sums, which a second kernel adds up in order.
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

constexpr int kThreads = 128;

// W 32-bit words (pairs of BF16): 8 by one access of 32 bytes, 4 by one of 16.
template <int W>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[W]) {
  if constexpr (W == 8) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
                   "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 v = *static_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}
template <int W>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[W]) {
  if constexpr (W == 8)
    stg256(p, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
  else
    *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// grad may be out: a thread reads an element before it writes it, and no other thread does either.
template <int ACT, int W>
__global__ void __launch_bounds__(kThreads) epilogue_backward_kernel(
    const uint32_t* grad, const uint32_t* z, int64_t M, int64_t pitch, uint32_t* out, float* partial,
    int64_t rows, uint32_t* amax) {
  constexpr int kRows = 2;
  pdl_wait();
  pdl_allow_next();
  const int64_t c = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * W;  // in words
  const int64_t first = (int64_t)blockIdx.y * rows, last = min(first + rows, M);
  uint64_t sum[W];
#pragma unroll
  for (int j = 0; j < W; j++) sum[j] = 0ull;
  uint32_t top = 0u;
  auto one = [&](const uint32_t (&g)[W], const uint32_t (&x)[W], int64_t at) {
    uint32_t o[W];
#pragma unroll
    for (int j = 0; j < W; j++) {
      const uint64_t d = f2_mul(f2_from_bf16x2(g[j]), activation_slope2<ACT>(f2_from_bf16x2(x[j])));
      sum[j] = f2_add(sum[j], d);
      const float2 f = f2_unpack(d);
      const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
      o[j] = *reinterpret_cast<const uint32_t*>(&p);
      top = hmax_abs2(top, o[j]);
    }
    store_words<W>(out + at, o);
  };
  if (c < pitch) {
    int64_t r = first;
    for (; r + kRows <= last; r += kRows) {
      uint32_t g[kRows][W], x[kRows][W];
#pragma unroll
      for (int i = 0; i < kRows; i++) {
        load_words<W>(grad + (r + i) * pitch + c, g[i]);
        load_words<W>(z + (r + i) * pitch + c, x[i]);
      }
#pragma unroll
      for (int i = 0; i < kRows; i++) one(g[i], x[i], (r + i) * pitch + c);
    }
    for (; r < last; r++) {
      uint32_t g[W], x[W];
      load_words<W>(grad + r * pitch + c, g);
      load_words<W>(z + r * pitch + c, x);
      one(g, x, r * pitch + c);
    }
    if (partial != nullptr) {
      float4* const to = reinterpret_cast<float4*>(partial + 2 * ((int64_t)blockIdx.y * pitch + c));
#pragma unroll
      for (int j = 0; j < W; j += 2) {
        const float2 a = f2_unpack(sum[j]), b = f2_unpack(sum[j + 1]);
        to[j / 2] = make_float4(a.x, a.y, b.x, b.y);
      }
    }
  }
  if (amax != nullptr) {
    top &= 0x7FFF7FFFu;
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(top << 16, top & 0xFFFF0000u));
    if ((threadIdx.x & 31) == 0 && m != 0u) atomicMax(amax, m);
  }
}

// Eight rows' sums are under way together, added up in their order.
__global__ void __launch_bounds__(kThreads) column_sum_kernel(const float* partial, int64_t rows, int64_t N,
                                                              float* out) {
  pdl_wait();
  pdl_allow_next();
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= N) return;
  float s = 0.0f;
  int64_t r = 0;
  for (; r + 8 <= rows; r += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = partial[(r + i) * N + c];
#pragma unroll
    for (int i = 0; i < 8; i++) s += v[i];
  }
  for (; r < rows; r++) s += partial[r * N + c];
  out[c] = s;
}

}  // namespace

cudaError_t launch_epilogue_backward(const void* grad, const void* preact, int64_t M, int64_t N,
                                     int32_t activation, void* grad_z, float* grad_bias, float* amax,
                                     float* partial, int sm_count, cudaStream_t s) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(grad) | reinterpret_cast<uintptr_t>(preact) |
                        reinterpret_cast<uintptr_t>(grad_z) | (uintptr_t)(N * 2);
  const bool wide = all % 32 == 0;
  const int64_t columns = kThreads * (wide ? 16 : 8), across = (N + columns - 1) / columns;
  // ranges of rows: eight CTAs an SM in all, at most the rows of the workspace
  int64_t down = (8 * sm_count) / across;
  if (down < 1) down = 1;
  if (down > kEpilogueMaxPartials) down = kEpilogueMaxPartials;
  if (down > M) down = M;
  const int64_t rows = (M + down - 1) / down;
  down = (M + rows - 1) / rows;
  const dim3 grid((unsigned)across, (unsigned)down), block(kThreads);
  auto run = [&](auto kernel8, auto kernel4) {
    return launch_pdl(wide ? kernel8 : kernel4, grid, block, 0, s, static_cast<const uint32_t*>(grad),
                      static_cast<const uint32_t*>(preact), M, N / 2, static_cast<uint32_t*>(grad_z),
                      grad_bias ? partial : nullptr, rows, reinterpret_cast<uint32_t*>(amax));
  };
  cudaError_t e;
  switch (activation) {
#define NVFP4_CASE(ACT) \
  case ACT: e = run(epilogue_backward_kernel<ACT, 8>, epilogue_backward_kernel<ACT, 4>); break;
    NVFP4_CASE(NVFP4_ACT_RELU)
    NVFP4_CASE(NVFP4_ACT_RELU2)
    NVFP4_CASE(NVFP4_ACT_GELU)
    NVFP4_CASE(NVFP4_ACT_SILU)
#undef NVFP4_CASE
    default: e = run(epilogue_backward_kernel<NVFP4_ACT_NONE, 8>, epilogue_backward_kernel<NVFP4_ACT_NONE, 4>);
  }
  if (e != cudaSuccess || grad_bias == nullptr) return e;
  return launch_pdl(column_sum_kernel, dim3((unsigned)((N + kThreads - 1) / kThreads)), block, 0, s,
                    (const float*)partial, down, N, grad_bias);
}

}  // namespace nvfp4
