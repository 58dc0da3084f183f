// Internal declarations of the matrix products of NVFP4 operands (gemm.cu, gemm_epilogue.cu and
// their C ABI in gemm_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "nvfp4.h"

namespace nvfp4 {

enum GemmMode : int32_t { kGemmDense = 0, kGemmGrouped = 1, kGemmWgrad = 2 };

// One call: out rows come from operand a, columns from operand b, both with K innermost.
//   dense    a [M][K], b [N][K]
//   grouped  a [M][K] with rows split by offsets, b [E][N][K]; z, bias and amax per expert
//   wgrad    a [M][K], b [N][K] with columns split by the padded counts of offsets; out [E][M][N]
struct GemmArgs {
  nvfp4_operand a, b;
  int64_t M, N, K;
  int32_t mode, E;
  const int32_t* offsets;
  int32_t activation, out_bytes, bias_bytes;
  const void* bias;
  const void* residual;
  void* preact;
  float* amax;
  void* out;
  void* workspace;        // 16-byte aligned, or null
  size_t workspace_bytes;
  uint32_t* status;
};
cudaError_t launch_gemm(const GemmArgs& g, int sm_count, cudaStream_t s);
cudaError_t prepare_gemm_kernels();
// bytes of workspace that spare the large tiles' kernel scales at any address
int64_t gemm_workspace(const GemmArgs& g);

constexpr int64_t kEpilogueMaxPartials = 512;  // rows of the bias gradient's partial sums
constexpr int64_t kEpilogueFewRows = 32;       // up to which there are none
cudaError_t launch_epilogue_backward(const void* grad, const void* preact, int64_t M, int64_t N,
                                     int32_t activation, void* grad_z, float* grad_bias, float* amax,
                                     float* partial, int sm_count, cudaStream_t s);

}  // namespace nvfp4
