// C ABI of the routing operators and of the operators with 8-bit checkpoints (declared in
// include/nvfp4.h): argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "nvfp4.h"
#include "nvfp4_device.cuh"
#include "aux_internal.h"
#include "nvfp4_internal.h"

#define NVFP4_EXPORT extern "C" __attribute__((visibility("default")))

using namespace nvfp4;

namespace {

// slots, rows and the blocks that are launched for them stay within 32 bits
constexpr int64_t kMaxRows = INT32_MAX - 65536;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

nvfp4_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return NVFP4_OK;
  (void)cudaGetLastError();
  return NVFP4_ERR_CUDA;
}

// Sizes shared by the routing calls; E = 1 where a call has no experts.
nvfp4_status check_route(int64_t T, int64_t H, int32_t K, int32_t E) {
  if (T < 0 || H < 0 || K < 1 || E < 1 || E > kMaxSegments) return NVFP4_ERR_INVALID_ARG;
  if (K > kMaxTopk) return NVFP4_ERR_UNSUPPORTED;
  if (H % 8 != 0 || H > INT32_MAX / 16 || T > kMaxRows / K) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

// Sizes shared by the checkpoint calls: rows of `width` elements in blocks of 32.
nvfp4_status check_rows(int64_t M, int64_t width) {
  if (M < 0 || width < 0) return NVFP4_ERR_INVALID_ARG;
  if (width % 32 != 0 || M > kMaxRows || width > INT32_MAX / 16) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

nvfp4_status check_segments(const int32_t* offsets, int32_t E) {
  if (offsets == nullptr) return E == 1 ? NVFP4_OK : NVFP4_ERR_INVALID_ARG;
  if (E < 1 || E > kMaxSegments) return NVFP4_ERR_INVALID_ARG;
  return aligned(offsets, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

__global__ void zero_kernel(float* p, int64_t n) {
  pdl_wait();
  pdl_allow_next();
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) p[i] = 0.0f;
}

// Clears n words by a kernel: a memset in the stream ends the overlap of the launches on both of
// its sides (with one before dispatch, 300 x 8 x 7168 takes 10.4 us, with this 7.2).
cudaError_t zero(void* p, int64_t n, cudaStream_t s) {
  if (p == nullptr || n == 0) return cudaSuccess;
  return launch_pdl(zero_kernel, dim3(1), dim3(256), 0, s, static_cast<float*>(p), n);
}

}  // namespace

cudaError_t nvfp4::zero_words(void* p, int64_t n, cudaStream_t s) { return zero(p, n, s); }

NVFP4_EXPORT nvfp4_status nvfp4_moe_plan(const void* expert_ids, int32_t id_bytes, int64_t T,
                                         int32_t K, int32_t E, int32_t* row_of_slot,
                                         int32_t* slot_of_row, int32_t* offsets, void* stream) {
  nvfp4_status st = check_route(T, 0, K, E);
  if (st != NVFP4_OK) return st;
  if (id_bytes != 4 && id_bytes != 8) return NVFP4_ERR_INVALID_ARG;
  const int64_t n = T * K;
  if (offsets == nullptr || (n > 0 && (expert_ids == nullptr || row_of_slot == nullptr ||
                                       slot_of_row == nullptr)))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(offsets, 4) || (n > 0 && (!aligned(expert_ids, (uintptr_t)id_bytes) ||
                                         !aligned(row_of_slot, 4) || !aligned(slot_of_row, 4))))
    return NVFP4_ERR_ALIGN;
  int sms = 0, ctas = 0;
  uint32_t* status = nullptr;
  if (!device_resources(&sms, &status, &ctas)) return NVFP4_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) return cuda_status(zero(offsets, E, s));
  return cuda_status(launch_moe_plan(expert_ids, id_bytes == 8, (int32_t)n, E, row_of_slot,
                                     slot_of_row, offsets, status, ctas, s));
}

NVFP4_EXPORT nvfp4_status nvfp4_moe_dispatch(const void* x, const int32_t* row_of_slot,
                                             const int32_t* offsets, int64_t T, int64_t H,
                                             int32_t K, int32_t E, void* packed, float* amax,
                                             void* stream) {
  nvfp4_status st = check_route(T, H, K, E);
  if (st != NVFP4_OK) return st;
  const bool empty = T * H == 0;
  if (!empty && (x == nullptr || row_of_slot == nullptr || offsets == nullptr || packed == nullptr))
    return NVFP4_ERR_INVALID_ARG;
  if ((!empty && (!aligned(x, 16) || !aligned(packed, 16) || !aligned(row_of_slot, 4) ||
                  !aligned(offsets, 4))) ||
      !aligned(amax, 4))
    return NVFP4_ERR_ALIGN;
  int sms = 0;
  uint32_t* status = nullptr;
  if (!device_resources(&sms, &status)) return NVFP4_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      !empty && moe_dispatch_clears_amax(T) ? cudaSuccess : zero(amax, E, s);
  if (e != cudaSuccess || empty) return cuda_status(e);
  return cuda_status(launch_moe_dispatch(x, row_of_slot, offsets, T, K, E, H / 8, packed, amax,
                                         status, sms, s));
}

// Combine (weights given) and the gradient of dispatch (weights null).
static nvfp4_status gather_sum(const void* rows, const float* weights, bool weighted,
                               const int32_t* row_of_slot, int64_t T, int64_t H, int32_t K,
                               void* out, void* stream) {
  nvfp4_status st = check_route(T, H, K, 1);
  if (st != NVFP4_OK) return st;
  if (T * H == 0) return NVFP4_OK;
  if (rows == nullptr || row_of_slot == nullptr || out == nullptr ||
      (weighted && weights == nullptr))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(rows, 16) || !aligned(out, 16) || !aligned(row_of_slot, 4) || !aligned(weights, 4))
    return NVFP4_ERR_ALIGN;
  int sms = 0;
  uint32_t* status = nullptr;
  if (!device_resources(&sms, &status)) return NVFP4_ERR_CUDA;
  return cuda_status(launch_moe_gather_sum(rows, weights, row_of_slot, T, K, H / 8, out, status,
                                           sms, static_cast<cudaStream_t>(stream)));
}

NVFP4_EXPORT nvfp4_status nvfp4_moe_dispatch_backward(const void* grad_packed,
                                                      const int32_t* row_of_slot, int64_t T,
                                                      int64_t H, int32_t K, void* grad_x,
                                                      void* stream) {
  return gather_sum(grad_packed, nullptr, false, row_of_slot, T, H, K, grad_x, stream);
}

NVFP4_EXPORT nvfp4_status nvfp4_moe_combine(const void* y, const float* weights,
                                            const int32_t* row_of_slot, int64_t T, int64_t H,
                                            int32_t K, void* out, void* stream) {
  return gather_sum(y, weights, true, row_of_slot, T, H, K, out, stream);
}

NVFP4_EXPORT nvfp4_status nvfp4_moe_combine_backward(const void* grad_out, const void* y,
                                                     const float* weights,
                                                     const int32_t* row_of_slot,
                                                     const int32_t* offsets, int64_t T, int64_t H,
                                                     int32_t K, int32_t E, void* grad_y,
                                                     float* grad_weights, void* stream) {
  nvfp4_status st = check_route(T, H, K, E);
  if (st != NVFP4_OK) return st;
  if (T == 0) return NVFP4_OK;
  if (grad_weights == nullptr ||
      (H > 0 && (grad_out == nullptr || y == nullptr || weights == nullptr ||
                 row_of_slot == nullptr || offsets == nullptr || grad_y == nullptr)))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(grad_weights, 4) ||
      (H > 0 && (!aligned(grad_out, 16) || !aligned(y, 16) || !aligned(grad_y, 16) ||
                 !aligned(weights, 4) || !aligned(row_of_slot, 4) || !aligned(offsets, 4))))
    return NVFP4_ERR_ALIGN;
  int sms = 0;
  uint32_t* status = nullptr;
  if (!device_resources(&sms, &status)) return NVFP4_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (H == 0) return cuda_status(zero(grad_weights, T * K, s));
  return cuda_status(launch_moe_combine_backward(grad_out, y, weights, row_of_slot, offsets, T, K,
                                                 E, H / 8, grad_y, grad_weights, status, sms, s));
}

NVFP4_EXPORT nvfp4_status nvfp4_swiglu_checkpoint(const void* h, int64_t M, int64_t F,
                                                  const int32_t* offsets, int32_t E, void* y,
                                                  uint8_t* codes, uint8_t* scales, float* amax,
                                                  void* stream) {
  nvfp4_status st = check_rows(M, F);
  if (st != NVFP4_OK || (st = check_segments(offsets, E)) != NVFP4_OK) return st;
  const bool empty = M * F == 0;
  if (!empty && (h == nullptr || y == nullptr || codes == nullptr || scales == nullptr))
    return NVFP4_ERR_INVALID_ARG;
  if ((!empty && (!aligned(h, 32) || !aligned(y, 32) || !aligned(codes, 16))) || !aligned(amax, 4))
    return NVFP4_ERR_ALIGN;
  int sms = 0;
  uint32_t* status = nullptr;
  if (!device_resources(&sms, &status)) return NVFP4_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = zero(amax, E, s);
  if (e != cudaSuccess || empty) return cuda_status(e);
  return cuda_status(launch_swiglu_checkpoint(h, M, F, offsets, E, y, codes, scales, amax, status,
                                              sms, s));
}

NVFP4_EXPORT nvfp4_status nvfp4_swiglu_checkpoint_backward(const void* grad_y,
                                                           const uint8_t* codes,
                                                           const uint8_t* scales, int64_t M,
                                                           int64_t F, const int32_t* offsets,
                                                           int32_t E, void* grad_h, void* stream) {
  nvfp4_status st = check_rows(M, F);
  if (st != NVFP4_OK || (st = check_segments(offsets, E)) != NVFP4_OK) return st;
  if (M * F == 0) return NVFP4_OK;
  if (grad_y == nullptr || codes == nullptr || scales == nullptr || grad_h == nullptr)
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(grad_y, 32) || !aligned(codes, 16) || !aligned(grad_h, 32)) return NVFP4_ERR_ALIGN;
  int sms = 0;
  uint32_t* status = nullptr;
  if (!device_resources(&sms, &status)) return NVFP4_ERR_CUDA;
  return cuda_status(launch_swiglu_checkpoint_backward(grad_y, codes, scales, M, F, offsets, E,
                                                       grad_h, status, sms,
                                                       static_cast<cudaStream_t>(stream)));
}

NVFP4_EXPORT nvfp4_status nvfp4_rmsnorm_checkpoint(const void* x, const void* weight, int64_t M,
                                                   int64_t N, float eps, float weight_bias, void* y,
                                                   uint8_t* codes, uint8_t* scales, float* rstd,
                                                   float* amax, void* stream) {
  nvfp4_status st = check_rows(M, N);
  if (st != NVFP4_OK) return st;
  if (amax == nullptr || !std::isfinite(eps) || !std::isfinite(weight_bias))
    return NVFP4_ERR_INVALID_ARG;
  if (N > kRmsMaxN) return NVFP4_ERR_UNSUPPORTED;
  const bool empty = M * N == 0;
  if (!empty && (x == nullptr || weight == nullptr || y == nullptr || codes == nullptr ||
                 scales == nullptr || rstd == nullptr))
    return NVFP4_ERR_INVALID_ARG;
  if ((!empty && (!aligned(x, 32) || !aligned(weight, 32) || !aligned(y, 32) ||
                  !aligned(codes, 16) || !aligned(rstd, 4))) ||
      !aligned(amax, 4))
    return NVFP4_ERR_ALIGN;
  int sms = 0;
  uint32_t* status = nullptr;
  if (!device_resources(&sms, &status)) return NVFP4_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = zero(amax, 1, s);
  if (e != cudaSuccess || empty) return cuda_status(e);
  RmsArgs a = {};
  a.M = M; a.N = N; a.eps = eps; a.bias = weight_bias;
  a.x = x; a.weight = weight; a.y = y; a.codes = codes; a.scales = scales; a.rstd = rstd;
  a.amax = amax; a.status = status;
  return cuda_status(launch_rmsnorm_checkpoint(a, sms, s));
}

NVFP4_EXPORT nvfp4_status nvfp4_rmsnorm_checkpoint_workspace(int64_t M, int64_t N, size_t* bytes) {
  if (bytes == nullptr) return NVFP4_ERR_INVALID_ARG;
  const nvfp4_status st = check_rows(M, N);
  if (st != NVFP4_OK) return st;
  if (N > kRmsMaxN) return NVFP4_ERR_UNSUPPORTED;
  *bytes = (size_t)(M < kRmsMaxPartials ? M : kRmsMaxPartials) * (size_t)N * 4;
  return NVFP4_OK;
}

NVFP4_EXPORT nvfp4_status nvfp4_rmsnorm_checkpoint_backward(
    const void* grad_y, const uint8_t* codes, const uint8_t* scales, const float* rstd,
    const void* weight, int64_t M, int64_t N, float weight_bias, const void* grad_residual,
    void* grad_x, float* grad_weight, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  nvfp4_status st = nvfp4_rmsnorm_checkpoint_workspace(M, N, &need);
  if (st != NVFP4_OK) return st;
  if (!std::isfinite(weight_bias) || (N > 0 && grad_weight == nullptr))
    return NVFP4_ERR_INVALID_ARG;
  const bool empty = M * N == 0;
  if (!empty && (grad_y == nullptr || codes == nullptr || scales == nullptr || rstd == nullptr ||
                 weight == nullptr || grad_x == nullptr || workspace == nullptr ||
                 workspace_bytes < need))
    return NVFP4_ERR_INVALID_ARG;
  if ((!empty && (!aligned(grad_y, 32) || !aligned(codes, 16) || !aligned(rstd, 4) ||
                  !aligned(weight, 32) || !aligned(grad_residual, 32) || !aligned(grad_x, 32) ||
                  !aligned(workspace, 16))) ||
      !aligned(grad_weight, 16))
    return NVFP4_ERR_ALIGN;
  int sms = 0;
  uint32_t* status = nullptr;
  if (!device_resources(&sms, &status)) return NVFP4_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) return cuda_status(zero(grad_weight, N, s));
  RmsArgs a = {};
  a.M = M; a.N = N; a.bias = weight_bias;
  a.grad = grad_y; a.codes = const_cast<uint8_t*>(codes); a.scales = const_cast<uint8_t*>(scales);
  a.rstd = const_cast<float*>(rstd); a.weight = weight; a.residual = grad_residual;
  a.grad_x = grad_x; a.grad_weight = grad_weight; a.partial = static_cast<float*>(workspace);
  a.status = status;
  return cuda_status(launch_rmsnorm_checkpoint_backward(a, sms, s));
}
