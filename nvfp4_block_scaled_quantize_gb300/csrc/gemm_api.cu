// C ABI of the matrix products (declared in include/nvfp4.h): argument checks and launches.
#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4.h"
#include "aux_internal.h"
#include "gemm_internal.h"
#include "nvfp4_internal.h"

#define NVFP4_EXPORT extern "C" __attribute__((visibility("default")))

using namespace nvfp4;

namespace {

constexpr int64_t kMaxDim = INT32_MAX - 65536;  // rows, columns and K stay within 32 bits

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

nvfp4_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return NVFP4_OK;
  (void)cudaGetLastError();
  return NVFP4_ERR_CUDA;
}

nvfp4_status check_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return NVFP4_ERR_INVALID_ARG;
  if (K % 32 != 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

// An operand of `rows` rows and K columns that the call reads; `experts` > 1: stacked.
nvfp4_status check_operand(const nvfp4_operand* o, int64_t rows, int64_t K, int32_t experts) {
  if (o == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (o->gscale == nullptr || (rows > 0 && K > 0 && (o->codes == nullptr || o->scales == nullptr)))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(o->gscale, 4)) return NVFP4_ERR_ALIGN;
  if (rows == 0 || K == 0) return NVFP4_OK;
  if (!aligned(o->codes, 16)) return NVFP4_ERR_ALIGN;
  if (rows > 1) {
    if (o->code_pitch < K / 2 || o->scale_pitch < K / 16) return NVFP4_ERR_SHAPE;
  }
  if (o->code_pitch < 0 || o->scale_pitch < 0 || o->code_pitch > (int64_t(1) << 38) ||
      o->scale_pitch > (int64_t(1) << 38))
    return NVFP4_ERR_SHAPE;
  if (o->code_pitch % 16 != 0) return NVFP4_ERR_ALIGN;
  if (experts > 1) {
    if (o->code_batch < K / 2 || o->scale_batch < K / 16 || o->code_batch > (int64_t(1) << 38) ||
        o->scale_batch > (int64_t(1) << 38))
      return NVFP4_ERR_SHAPE;
    if (o->code_batch % 16 != 0) return NVFP4_ERR_ALIGN;
  }
  return NVFP4_OK;
}

nvfp4_status check_workspace(const void* workspace, size_t bytes) {
  if (workspace == nullptr && bytes != 0) return NVFP4_ERR_INVALID_ARG;
  return aligned(workspace, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

nvfp4_status check_epilogue(const nvfp4_epilogue* e, const void* out, bool empty) {
  if (e == nullptr || (e->out_bytes != 2 && e->out_bytes != 4) || e->activation < NVFP4_ACT_NONE ||
      e->activation > NVFP4_ACT_SILU || (e->bias && e->bias_bytes != 2 && e->bias_bytes != 4))
    return NVFP4_ERR_INVALID_ARG;
  if (!empty && out == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(out, (uintptr_t)e->out_bytes) || !aligned(e->residual, (uintptr_t)e->out_bytes) ||
      !aligned(e->preact, 2) || !aligned(e->amax, 4) ||
      (e->bias && !aligned(e->bias, (uintptr_t)e->bias_bytes)))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

void take_epilogue(GemmArgs& g, const nvfp4_epilogue& e) {
  g.activation = e.activation;
  g.out_bytes = e.out_bytes;
  g.bias_bytes = e.bias_bytes;
  g.bias = e.bias;
  g.residual = e.residual;
  g.preact = e.preact;
  g.amax = e.amax;
}

}  // namespace

NVFP4_EXPORT nvfp4_status nvfp4_gemm_workspace(const nvfp4_operand* a, const nvfp4_operand* b, int64_t M,
                                               int64_t N, int64_t K, int32_t E, size_t* bytes) {
  if (bytes == nullptr || E < 1 || E > kMaxSegments) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = check_sizes(M, N, K);
  if (st != NVFP4_OK || (st = check_operand(a, M, K, 1)) != NVFP4_OK ||
      (st = check_operand(b, N, K, E)) != NVFP4_OK)
    return st;
  GemmArgs g = {};
  g.a = *a, g.b = *b;
  g.M = M, g.N = N, g.K = K, g.mode = kGemmGrouped, g.E = E;
  *bytes = (size_t)gemm_workspace(g);
  return NVFP4_OK;
}

NVFP4_EXPORT nvfp4_status nvfp4_gemm(const nvfp4_operand* a, const nvfp4_operand* b, int64_t M,
                                     int64_t N, int64_t K, const nvfp4_epilogue* epilogue, void* out,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  nvfp4_status st = check_sizes(M, N, K);
  const bool empty = M == 0 || N == 0;
  if (st != NVFP4_OK || (st = check_operand(a, M, K, 1)) != NVFP4_OK ||
      (st = check_operand(b, N, K, 1)) != NVFP4_OK ||
      (st = check_epilogue(epilogue, out, empty)) != NVFP4_OK ||
      (st = check_workspace(workspace, workspace_bytes)) != NVFP4_OK)
    return st;
  int sms = 0;
  uint32_t* status = nullptr;
  if (!device_basics(&sms, &status, true)) return NVFP4_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = zero_words(epilogue->amax, 1, s);
  if (e != cudaSuccess || empty) return cuda_status(e);
  GemmArgs g = {};
  g.a = *a, g.b = *b;
  g.M = M, g.N = N, g.K = K, g.mode = kGemmDense, g.E = 1;
  take_epilogue(g, *epilogue);
  g.out = out, g.workspace = workspace, g.workspace_bytes = workspace_bytes, g.status = status;
  return cuda_status(launch_gemm(g, sms, s));
}

NVFP4_EXPORT nvfp4_status nvfp4_gemm_grouped(const nvfp4_operand* a, const nvfp4_operand* b,
                                             const int32_t* offsets, int32_t E, int64_t T, int64_t N,
                                             int64_t K, const nvfp4_epilogue* epilogue, void* out,
                                             void* workspace, size_t workspace_bytes, void* stream) {
  nvfp4_status st = check_sizes(T, N, K);
  const bool empty = T == 0 || N == 0;
  if (st != NVFP4_OK) return st;
  if (E < 1 || E > kMaxSegments || offsets == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(offsets, 4)) return NVFP4_ERR_ALIGN;
  if ((st = check_operand(a, T, K, 1)) != NVFP4_OK || (st = check_operand(b, N, K, E)) != NVFP4_OK ||
      (st = check_epilogue(epilogue, out, empty)) != NVFP4_OK ||
      (st = check_workspace(workspace, workspace_bytes)) != NVFP4_OK)
    return st;
  int sms = 0;
  uint32_t* status = nullptr;
  if (!device_basics(&sms, &status, true)) return NVFP4_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = zero_words(epilogue->amax, E, s);
  if (e != cudaSuccess || empty) return cuda_status(e);
  GemmArgs g = {};
  g.a = *a, g.b = *b;
  g.M = T, g.N = N, g.K = K, g.mode = kGemmGrouped, g.E = E, g.offsets = offsets;
  take_epilogue(g, *epilogue);
  g.out = out, g.workspace = workspace, g.workspace_bytes = workspace_bytes, g.status = status;
  return cuda_status(launch_gemm(g, sms, s));
}

NVFP4_EXPORT nvfp4_status nvfp4_gemm_grouped_wgrad(const nvfp4_operand* a, const nvfp4_operand* b,
                                                   const int32_t* offsets, int32_t E, int64_t M,
                                                   int64_t N, int64_t capacity, int32_t out_bytes,
                                                   int32_t accumulate, void* out, void* workspace,
                                                   size_t workspace_bytes, void* stream) {
  nvfp4_status st = check_sizes(M, N, capacity);
  const bool empty = M == 0 || N == 0;
  if (st != NVFP4_OK) return st;
  if (E < 1 || E > kMaxSegments || offsets == nullptr || (accumulate != 0 && accumulate != 1))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(offsets, 4)) return NVFP4_ERR_ALIGN;
  nvfp4_epilogue ep = {};
  ep.out_bytes = out_bytes;
  if ((st = check_operand(a, M, capacity, 1)) != NVFP4_OK ||
      (st = check_operand(b, N, capacity, 1)) != NVFP4_OK ||
      (st = check_epilogue(&ep, out, empty)) != NVFP4_OK ||
      (st = check_workspace(workspace, workspace_bytes)) != NVFP4_OK)
    return st;
  if (accumulate) ep.residual = out;
  if (empty) return NVFP4_OK;
  int sms = 0;
  uint32_t* status = nullptr;
  if (!device_basics(&sms, &status, true)) return NVFP4_ERR_CUDA;
  GemmArgs g = {};
  g.a = *a, g.b = *b;
  g.M = M, g.N = N, g.K = capacity, g.mode = kGemmWgrad, g.E = E, g.offsets = offsets;
  take_epilogue(g, ep);
  g.out = out, g.workspace = workspace, g.workspace_bytes = workspace_bytes, g.status = status;
  return cuda_status(launch_gemm(g, sms, static_cast<cudaStream_t>(stream)));
}

NVFP4_EXPORT nvfp4_status nvfp4_gemm_epilogue_backward_workspace(int64_t M, int64_t N, size_t* bytes) {
  if (bytes == nullptr || M < 0 || N < 0) return NVFP4_ERR_INVALID_ARG;
  if (M > kMaxDim || N > kMaxDim) return NVFP4_ERR_SHAPE;
  *bytes = M <= kEpilogueFewRows ? 0 : (size_t)(M < kEpilogueMaxPartials ? M : kEpilogueMaxPartials) * (size_t)N * 4;
  return NVFP4_OK;
}

NVFP4_EXPORT nvfp4_status nvfp4_gemm_epilogue_backward(const void* grad_out, const void* preact, int64_t M,
                                                       int64_t N, int32_t activation, void* grad_preact,
                                                       float* grad_bias, float* amax, void* workspace,
                                                       size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const nvfp4_status st = nvfp4_gemm_epilogue_backward_workspace(M, N, &need);
  if (st != NVFP4_OK) return st;
  if (activation < NVFP4_ACT_NONE || activation > NVFP4_ACT_SILU) return NVFP4_ERR_INVALID_ARG;
  const bool empty = M == 0 || N == 0;
  if (!empty && (grad_out == nullptr || preact == nullptr || grad_preact == nullptr ||
                 (grad_bias != nullptr && need > 0 && (workspace == nullptr || workspace_bytes < need))))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(grad_out, 16) || !aligned(preact, 16) || !aligned(grad_preact, 16) ||
      !aligned(grad_bias, 16) || !aligned(amax, 4) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  int sms = 0;
  uint32_t* status = nullptr;
  if (!device_basics(&sms, &status)) return NVFP4_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = zero_words(amax, 1, s);
  if (e == cudaSuccess && empty) e = zero_words(grad_bias, N, s);
  if (e != cudaSuccess || empty) return cuda_status(e);
  return cuda_status(launch_epilogue_backward(grad_out, preact, M, N, activation, grad_preact, grad_bias,
                                              amax, static_cast<float*>(workspace), sms, s));
}
