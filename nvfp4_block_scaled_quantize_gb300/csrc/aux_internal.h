// Internal declarations of the library's kernels other than the tile kernel (not part of the
// C ABI): MX quantization, the RMSNorm producer, token routing, the operators with 8-bit
// checkpoints, the flat amax, the scale swizzle and dequantization. Kept apart from
// nvfp4_internal.h, whose contents the tile kernel depends on.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace nvfp4 {

// ---- MX formats (mx_kernel.cu): 32-element blocks, E8M0 scales, no tensor scale ----
// A warp quantizes 32 x 128 units alone, kMxStages of them in flight in its own ring; a unit is
// two TMA boxes of 32 rows x 64 BF16 columns (128-byte rows, 128-byte swizzle). Its codes are
// staged in kMxOutBytes of shared memory per warp and leave by TMA stores.
constexpr int kMxUnitM = 32;
constexpr int kMxUnitN = 128;
constexpr int kMxWarps = 8;
constexpr int kMxStages = 2;
constexpr int kMxOutBytes = 8192;  // row codes, then column codes: 4 KiB each (FP8)
constexpr int kMxSmemBytes = kMxWarps * (kMxStages * (kMxUnitM * kMxUnitN * 2) + kMxOutBytes) +
                             2 * kMxWarps * kMxUnitN + kMxWarps * kMxStages * 8 + 1024;

struct MxArgs {
  CUtensorMap tmap;        // x as BF16 [rows][cols], box {64, 32}, 128-byte swizzle
  CUtensorMap tmap_row;    // row codes as bytes, box {128 (FP4: 64), 32}, swizzle span = row
  CUtensorMap tmap_col;    // column codes as bytes {M, N/4, 4}, box {32 (FP4: 16), 32, 4}
  int64_t rows, cols;
  uint8_t* row_codes;      // [rows][cols] FP8 or [rows][cols / 2] FP4
  uint8_t* row_scales;     // [rows][cols / 32] E8M0
  uint8_t* col_codes;      // [cols][rows] FP8 or [cols][rows / 2] FP4
  uint8_t* col_scales;     // [cols][rows / 32] E8M0
  uint32_t* status;
};
// fmt: 0 = E4M3, 1 = E5M2, 2 = E2M1
cudaError_t launch_mx_quantize(int fmt, bool row, bool col, const MxArgs& args, int grid,
                               cudaStream_t s);
cudaError_t prepare_mx_kernels();
cudaError_t launch_mx_dequantize(int fmt, const uint8_t* codes, const uint8_t* scales, int64_t R,
                                 int64_t C, float* out, int grid, cudaStream_t s);

// RMSNorm producer with the amax in its epilogue (producer.cu): y and an atomic max of |y|
// into *amax (zeroed by the caller); rmsnorm_rows_per_cta() rows per CTA.
cudaError_t launch_rmsnorm_amax(const void* x, const void* w, int64_t M, int64_t N, float eps,
                                float bias, void* y, float* amax, int grid, cudaStream_t s);
int rmsnorm_rows_per_cta();

// ---- token routing (moe_route.cu) ----
constexpr int kMaxTopk = 32;  // choices of a token: one warp loads a token's rows
// rows of `nv` 16-byte vectors; amax may be null, and the caller zeroes it unless
// moe_dispatch_clears_amax(T)
bool moe_dispatch_clears_amax(int64_t T);
// plan_ctas: the largest cluster of the plan that the current device holds
cudaError_t prepare_moe_kernels(int* plan_ctas);
cudaError_t launch_moe_plan(const void* ids, bool wide, int32_t n, int32_t E, int32_t* row_of_slot,
                            int32_t* slot_of_row, int32_t* offsets, uint32_t* status,
                            int plan_ctas, cudaStream_t s);
cudaError_t launch_moe_dispatch(const void* x, const int32_t* row_of_slot, const int32_t* offsets,
                                int64_t T, int32_t K, int32_t E, int64_t nv, void* packed,
                                float* amax, uint32_t* status, int sm_count, cudaStream_t s);
// weights null: all 1 (the gradient of dispatch)
cudaError_t launch_moe_gather_sum(const void* y, const float* weights, const int32_t* row_of_slot,
                                  int64_t T, int32_t K, int64_t nv, void* out, uint32_t* status,
                                  int sm_count, cudaStream_t s);
cudaError_t launch_moe_combine_backward(const void* grad, const void* y, const float* weights,
                                        const int32_t* row_of_slot, const int32_t* offsets,
                                        int64_t T, int32_t K, int32_t E, int64_t nv, void* grad_y,
                                        float* grad_w, uint32_t* status, int sm_count,
                                        cudaStream_t s);

// ---- operators with 8-bit checkpoints (checkpoint.cu) ----
cudaError_t prepare_checkpoint_kernels();
cudaError_t launch_swiglu_checkpoint(const void* h, int64_t M, int64_t F, const int32_t* offsets,
                                     int32_t E, void* y, void* codes, uint8_t* scales, float* amax,
                                     uint32_t* status, int sm_count, cudaStream_t s);
cudaError_t launch_swiglu_checkpoint_backward(const void* grad, const void* codes,
                                              const uint8_t* scales, int64_t M, int64_t F,
                                              const int32_t* offsets, int32_t E, void* grad_h,
                                              uint32_t* status, int sm_count, cudaStream_t s);
// a row stays in one CTA from the sum to the output: in registers (forward; backward as xh and g up
// to 8192 columns), or in the ring's shared memory (backward above that)
constexpr int64_t kRmsMaxN = 32768;
constexpr int64_t kRmsMaxPartials = 512;  // rows of the weight gradient's partial sums
struct RmsArgs {
  int64_t M, N;
  float eps, bias;
  const void *x, *weight, *grad, *residual;  // residual may be null
  void *y, *codes, *grad_x;
  uint8_t* scales;
  float *rstd, *amax, *partial, *grad_weight;
  uint32_t* status;
};
cudaError_t launch_rmsnorm_checkpoint(const RmsArgs& a, int sm_count, cudaStream_t s);
cudaError_t launch_rmsnorm_checkpoint_backward(const RmsArgs& a, int sm_count, cudaStream_t s);

// The current device's SM count, status word and largest cluster of the plan, with the kernels of
// these two groups set up (nvfp4_api.cu); false when a CUDA call failed.
bool device_resources(int* sm_count, uint32_t** status, int* plan_ctas = nullptr);
// The same without those kernels' set-up, with the matrix products' where `gemm` is set.
bool device_basics(int* sm_count, uint32_t** status, bool gemm = false);
int setup_fault();  // nvfp4_debug_setup_fault
// cuTensorMapEncodeTiled; set once a call above has succeeded (nvfp4_api.cu)
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled();
// Clears n 32-bit words in stream order, by a kernel (moe_checkpoint_api.cu); p may be null.
cudaError_t zero_words(void* p, int64_t n, cudaStream_t s);

cudaError_t launch_amax_flat(const void* x, int64_t n_elems, float* out0, float* out1, int grid,
                             cudaStream_t s);
cudaError_t launch_swizzle_scales(const uint8_t* scales, int64_t R, int64_t C, uint8_t* out,
                                  int grid, cudaStream_t s);
cudaError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, const float* gscale,
                              int64_t R, int64_t C, bool inverse_rht, uint32_t sign_mask,
                              bool out_bf16, void* out, int grid, cudaStream_t s);

}  // namespace nvfp4
