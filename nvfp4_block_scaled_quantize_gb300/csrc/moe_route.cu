// Token routing around the grouped quantizer: the plan (a stable counting sort of the (token,
// choice) slots by expert), the dispatch of token rows into that packed order, the weighted sum
// of expert outputs back into token order, and the gradients of both.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4_device.cuh"
#include "aux_internal.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanBatch = 8;  // groups of 32 slots whose ids a warp loads together
constexpr int kRouteThreads = 128;
constexpr uint32_t kBadRoute = 0x4u;  // NVFP4_DEVICE_BAD_ROUTE

// ---- plan --------------------------------------------------------------------------------

// Every warp owns a run of consecutive slots, every CTA of the cluster consecutive runs. Counts
// per (warp, expert) are summed over the warps, the CTAs' totals are exchanged through
// distributed shared memory, and the exclusive prefix (expert, CTA, warp) is the row of the first
// slot of that expert in that run; a second walk over the run hands the rows out in slot order.
// So the order is that of a stable sort, whatever the timing.
template <typename Id>
__global__ void __launch_bounds__(kPlanThreads) moe_plan_kernel(
    const Id* __restrict__ ids, int32_t n, int32_t run, int32_t E, int32_t* row_of_slot,
    int32_t* slot_of_row, int32_t* offsets, uint32_t* status) {
  namespace cg = cooperative_groups;
  __shared__ uint32_t hist[kPlanWarps][kMaxSegments];
  __shared__ uint32_t total[kMaxSegments];
  __shared__ uint32_t scan[kMaxSegments / 32];
  __shared__ uint32_t live;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kPlanWarps * kMaxSegments; i += kPlanThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_allow_next();

  const int64_t first = ((int64_t)rank * kPlanWarps + warp) * run;
  const int32_t begin = (int32_t)(first < n ? first : n);
  const int32_t end = n - begin < run ? n : begin + run;
  bool bad = false;
  for (int32_t s0 = begin; s0 < end; s0 += 32 * kPlanBatch) {
    Id id[kPlanBatch];
#pragma unroll
    for (int j = 0; j < kPlanBatch; j++) {
      const int32_t s = s0 + 32 * j + lane;
      id[j] = s < end ? ids[s] : (Id)-1;
    }
#pragma unroll
    for (int j = 0; j < kPlanBatch; j++) {
      if (id[j] >= 0 && id[j] < E)
        atomicAdd(&hist[warp][(int)id[j]], 1u);
      else if (id[j] >= E)
        bad = true;
    }
  }
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(status, kBadRoute);
  __syncthreads();
  if (tid < kMaxSegments) {  // counts -> exclusive prefixes over this CTA's warps
    uint32_t sum = 0;
#pragma unroll 8
    for (int w = 0; w < kPlanWarps; w++) {
      const uint32_t c = hist[w][tid];
      hist[w][tid] = sum;
      sum += c;
    }
    total[tid] = sum;
  }
  cluster.sync();
  uint32_t before = 0, all = 0, incl = 0;
  if (tid < kMaxSegments) {
    for (int c = 0; c < ctas; c++) {
      const uint32_t v = cluster.map_shared_rank(total, c)[tid];
      if (c < rank) before += v;
      all += v;
    }
    incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
  }
  __syncthreads();
  if (tid < kMaxSegments) {
    for (int w = 0; w < warp; w++) incl += scan[w];
    if (rank == 0 && tid < E) offsets[tid] = (int32_t)incl;
    if (tid == kMaxSegments - 1) live = incl;
    const uint32_t base = incl - all + before;
#pragma unroll 8
    for (int w = 0; w < kPlanWarps; w++) hist[w][tid] += base;
  }
  __syncthreads();
  // the same number of steps for every lane: the match below takes the whole warp
  for (int32_t s0 = begin; s0 < end; s0 += 32 * kPlanBatch) {
    int32_t e[kPlanBatch];
#pragma unroll
    for (int j = 0; j < kPlanBatch; j++) {
      const int32_t s = s0 + 32 * j + lane;
      const Id id = s < end ? ids[s] : (Id)-1;
      e[j] = id >= 0 && id < E ? (int32_t)id : -1;
    }
#pragma unroll
    for (int j = 0; j < kPlanBatch; j++) {
      const int32_t s = s0 + 32 * j + lane;
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, e[j]);
      const int before_me = __popc(peers & ((1u << lane) - 1u));
      int32_t row = -1;
      if (e[j] >= 0) row = (int32_t)(hist[warp][e[j]] + before_me);
      __syncwarp();
      if (e[j] >= 0 && before_me == 0) hist[warp][e[j]] += __popc(peers);
      __syncwarp();
      if (s < end) {
        row_of_slot[s] = row;
        if (row >= 0) slot_of_row[row] = s;
      }
    }
  }
  for (int64_t r = (int64_t)live + rank * kPlanThreads + tid; r < n;
       r += (int64_t)ctas * kPlanThreads)
    slot_of_row[r] = -1;
  cluster.sync();  // `total` stays until every CTA has read it
}

// ---- rows of a token ---------------------------------------------------------------------

// The token's rows that are held, in the order of its choices; whole CTA calls it, warp 0 works.
struct TokenRows {
  int32_t row[kMaxTopk];
  int32_t slot[kMaxTopk];
  int32_t count;
};

__device__ __forceinline__ void load_token_rows(TokenRows& r, const int32_t* row_of_slot,
                                                int64_t token, int32_t K, int64_t P,
                                                uint32_t* status) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int32_t row = lane < K ? row_of_slot[token * K + lane] : -1;
    if (row >= P) {
      atomicOr(status, kBadRoute);
      row = -1;
    }
    const uint32_t held = __ballot_sync(0xFFFFFFFFu, row >= 0);
    if (row >= 0) {
      const int at = __popc(held & ((1u << lane) - 1u));
      r.row[at] = row;
      r.slot[at] = lane;
    }
    if (lane == 0) r.count = __popc(held);
  }
}

__device__ __forceinline__ int64_t live_rows(const int32_t* offsets, int32_t E, int64_t P) {
  const int64_t v = offsets[E - 1];
  return v < 0 ? 0 : (v < P ? v : P);
}

// ---- dispatch ----------------------------------------------------------------------------

// grid.x: tokens, grid.y: ranges of `span` 16-byte vectors of a row.
__global__ void __launch_bounds__(kRouteThreads) moe_dispatch_kernel(
    const uint4* __restrict__ x, const int32_t* __restrict__ row_of_slot,
    const int32_t* __restrict__ offsets, int32_t K, int32_t E, int64_t nv, int64_t span,
    uint4* packed, uint32_t* amax, uint32_t* status) {
  __shared__ TokenRows rows;
  __shared__ int32_t ends[kMaxSegments];
  __shared__ uint32_t red[kRouteThreads / 32];
  pdl_wait();
  pdl_allow_next();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t token = blockIdx.x, P = (int64_t)gridDim.x * K;
  const int64_t v0 = (int64_t)blockIdx.y * span, v1 = v0 + span < nv ? v0 + span : nv;
  load_token_rows(rows, row_of_slot, token, K, P, status);
  for (int e = tid; e < E; e += kRouteThreads) ends[e] = offsets[e];
  __syncthreads();
  const int count = rows.count;
  uint32_t m = 0;
  for (int64_t v = v0 + tid; v < v1; v += kRouteThreads) {
    const uint4 q = x[token * nv + v];
    m = vmax2(m, vmax2(vmax2(abs2(q.x), abs2(q.y)), vmax2(abs2(q.z), abs2(q.w))));
    for (int k = 0; k < count; k++) packed[rows.row[k] * nv + v] = q;
  }
  m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  if (amax != nullptr && tid < count) {
    for (int w = 0; w < kRouteThreads / 32; w++) m = max(m, red[w]);
    const int32_t row = rows.row[tid];
    int lo = 0, hi = E;  // the expert of the row: the first whose end is past it
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ends[mid] > row) hi = mid; else lo = mid + 1;
    }
    if (lo < E) atomicMax(amax + lo, m << 16);
  }
  int64_t live = ends[E - 1];
  live = live < 0 ? 0 : live;
  for (int64_t r = live + token; r < P; r += gridDim.x)
    for (int64_t v = v0 + tid; v < v1; v += kRouteThreads)
      packed[r * nv + v] = make_uint4(0u, 0u, 0u, 0u);
}

// ---- combine and the gradient of dispatch ------------------------------------------------

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// out[t] = sum over the token's held rows of w * y[row], in the order of its choices, in binary32.
template <bool WEIGHTED>
__global__ void __launch_bounds__(kRouteThreads) moe_gather_sum_kernel(
    const uint4* __restrict__ y, const float* __restrict__ weights,
    const int32_t* __restrict__ row_of_slot, int32_t K, int64_t nv, int64_t span, uint4* out,
    uint32_t* status) {
  __shared__ TokenRows rows;
  pdl_wait();
  pdl_allow_next();
  const int64_t token = blockIdx.x, P = (int64_t)gridDim.x * K;
  const int64_t v0 = (int64_t)blockIdx.y * span, v1 = v0 + span < nv ? v0 + span : nv;
  load_token_rows(rows, row_of_slot, token, K, P, status);
  __syncthreads();
  const int count = rows.count;
  for (int64_t v = v0 + threadIdx.x; v < v1; v += kRouteThreads) {
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int k = 0; k < count; k++) {
      const uint4 q = y[rows.row[k] * nv + v];
      const uint32_t e[4] = {q.x, q.y, q.z, q.w};
      const float w = WEIGHTED ? weights[token * K + rows.slot[k]] : 1.0f;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        acc[2 * i] = __fmaf_rn(w, bf16_lo(e[i]), acc[2 * i]);
        acc[2 * i + 1] = __fmaf_rn(w, bf16_hi(e[i]), acc[2 * i + 1]);
      }
    }
    out[token * nv + v] = make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                                     pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7]));
  }
}

// ---- the gradient of combine -------------------------------------------------------------

// grad_y[row] = w * grad[t] and grad_w[t, k] = <grad[t], y[row]>: one CTA per token, kGroup of
// its rows at a time; rows past the last expert's end become zero.
constexpr int kGroup = 8;
__global__ void __launch_bounds__(kRouteThreads) moe_combine_backward_kernel(
    const uint4* __restrict__ grad, const uint4* __restrict__ y, const float* __restrict__ weights,
    const int32_t* __restrict__ row_of_slot, const int32_t* __restrict__ offsets, int32_t K,
    int32_t E, int64_t nv, uint4* grad_y, float* grad_w, uint32_t* status) {
  __shared__ TokenRows rows;
  __shared__ float red[kRouteThreads / 32][kGroup];
  pdl_wait();
  pdl_allow_next();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t token = blockIdx.x, P = (int64_t)gridDim.x * K;
  load_token_rows(rows, row_of_slot, token, K, P, status);
  if (tid < K) grad_w[token * K + tid] = 0.0f;  // the dropped slots keep it
  __syncthreads();
  const int count = rows.count;
  for (int k0 = 0; k0 < count; k0 += kGroup) {
    float dot[kGroup], w[kGroup];
#pragma unroll
    for (int j = 0; j < kGroup; j++) {
      dot[j] = 0.0f;
      w[j] = k0 + j < count ? weights[token * K + rows.slot[k0 + j]] : 0.0f;
    }
    for (int64_t v = tid; v < nv; v += kRouteThreads) {
      const uint4 g = grad[token * nv + v];
      const uint32_t ge[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int j = 0; j < kGroup; j++) {
        if (k0 + j < count) {
          const int64_t at = rows.row[k0 + j] * nv + v;
          const uint4 q = y[at];
          const uint32_t qe[4] = {q.x, q.y, q.z, q.w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            dot[j] = __fmaf_rn(bf16_lo(ge[i]), bf16_lo(qe[i]), dot[j]);
            dot[j] = __fmaf_rn(bf16_hi(ge[i]), bf16_hi(qe[i]), dot[j]);
            o[i] = pack_bf16(__fmul_rn(w[j], bf16_lo(ge[i])), __fmul_rn(w[j], bf16_hi(ge[i])));
          }
          grad_y[at] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kGroup; j++) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
      if (lane == 0) red[warp][j] = dot[j];
    }
    __syncthreads();
    if (tid < kGroup && k0 + tid < count) {
      float s = red[0][tid];
      for (int i = 1; i < kRouteThreads / 32; i++) s += red[i][tid];
      grad_w[token * K + rows.slot[k0 + tid]] = s;
    }
    __syncthreads();
  }
  for (int64_t r = live_rows(offsets, E, P) + token; r < P; r += gridDim.x)
    for (int64_t v = tid; v < nv; v += kRouteThreads)
      grad_y[r * nv + v] = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace

cudaError_t prepare_moe_kernels() {
  cudaError_t e = cudaSuccess, r;
  if ((r = cudaFuncSetAttribute(moe_plan_kernel<int32_t>,
                                cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
    e = r;
  if ((r = cudaFuncSetAttribute(moe_plan_kernel<int64_t>,
                                cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
    e = r;
  return e;
}

cudaError_t launch_moe_plan(const void* ids, bool wide, int32_t n, int32_t E, int32_t* row_of_slot,
                            int32_t* slot_of_row, int32_t* offsets, uint32_t* status,
                            cudaStream_t s) {
  const int ctas = n <= 4096 ? 1 : 16;
  const int64_t warps = (int64_t)ctas * kPlanWarps;
  const int32_t run = (int32_t)((n + warps * 32 - 1) / (warps * 32) * 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (wide)
    return cudaLaunchKernelEx(&cfg, moe_plan_kernel<int64_t>, static_cast<const int64_t*>(ids), n,
                              run, E, row_of_slot, slot_of_row, offsets, status);
  return cudaLaunchKernelEx(&cfg, moe_plan_kernel<int32_t>, static_cast<const int32_t*>(ids), n,
                            run, E, row_of_slot, slot_of_row, offsets, status);
}

// Ranges of a row: whole rows when there are tokens enough for every SM, else 128 vectors each.
static int64_t row_span(int64_t tokens, int64_t nv, int sm_count) {
  return tokens >= 4 * (int64_t)sm_count ? nv : kRouteThreads;
}

cudaError_t launch_moe_dispatch(const void* x, const int32_t* row_of_slot, const int32_t* offsets,
                                int64_t T, int32_t K, int32_t E, int64_t nv, void* packed,
                                float* amax, uint32_t* status, int sm_count, cudaStream_t s) {
  const int64_t span = row_span(T, nv, sm_count);
  return launch_pdl(moe_dispatch_kernel, dim3((unsigned)T, (unsigned)((nv + span - 1) / span)),
                    dim3(kRouteThreads), 0, s, static_cast<const uint4*>(x), row_of_slot, offsets,
                    K, E, nv, span, static_cast<uint4*>(packed),
                    reinterpret_cast<uint32_t*>(amax), status);
}

cudaError_t launch_moe_gather_sum(const void* y, const float* weights, const int32_t* row_of_slot,
                                  int64_t T, int32_t K, int64_t nv, void* out, uint32_t* status,
                                  int sm_count, cudaStream_t s) {
  const int64_t span = row_span(T, nv, sm_count);
  const dim3 grid((unsigned)T, (unsigned)((nv + span - 1) / span));
  return launch_pdl(weights ? moe_gather_sum_kernel<true> : moe_gather_sum_kernel<false>, grid,
                    dim3(kRouteThreads), 0, s, static_cast<const uint4*>(y), weights, row_of_slot,
                    K, nv, span, static_cast<uint4*>(out), status);
}

cudaError_t launch_moe_combine_backward(const void* grad, const void* y, const float* weights,
                                        const int32_t* row_of_slot, const int32_t* offsets,
                                        int64_t T, int32_t K, int32_t E, int64_t nv, void* grad_y,
                                        float* grad_w, uint32_t* status, cudaStream_t s) {
  return launch_pdl(moe_combine_backward_kernel, dim3((unsigned)T), dim3(kRouteThreads), 0, s,
                    static_cast<const uint4*>(grad), static_cast<const uint4*>(y), weights,
                    row_of_slot, offsets, K, E, nv, static_cast<uint4*>(grad_y), grad_w, status);
}

}  // namespace nvfp4
