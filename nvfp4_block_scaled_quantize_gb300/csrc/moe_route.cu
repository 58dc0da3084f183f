// Token routing around the grouped quantizer: the plan (a stable counting sort of the (token,
// choice) slots by expert), the dispatch of token rows into that packed order, the weighted sum
// of expert outputs back into token order, and the gradients of both.
//
// The plan is bound by the shared memory and the stores of the 16 SMs that one cluster has (14.9 us
// at 262144 slots, whose bytes would take 0.5 us; 25.0 at 524288, 42.0 at 1048576): one launch
// without scratch memory, whatever the size. The other four are bound by DRAM: at the measured copy
// rate of 6787 GB/s their bytes take 97% of dispatch's time (4096 x 8 rows of 7168, 80.1 us), 98%
// of combine's (8192 x 4 of 4096, 50.6 us), 98% of its gradient's (4096 x 8 of 7168, 148.0 us) and
// 81% (3001 x 6 of 2056) to 100% of the gradient of dispatch's. Dispatch of many rows of 129 to
// about 256 vectors is bound by its maxima, one atomic a slot: 16384 x 8 rows of 130 vectors take
// 74.6 us with 64 experts (60%), of 192 83.0 (80%), of 256 96.4 (92%).
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
constexpr int kPlanMaxCtas = 16;  // one cluster of the opt-in size
constexpr int kPlanPortableCtas = 8;  // where that does not fit
constexpr int kPlanMaxRun = 832;  // slots of a warp's run that is sorted in shared memory
constexpr int kPlanBatch = 8;  // groups of 32 slots whose ids a warp loads together
constexpr int kRouteThreads = 128;
constexpr uint32_t kBadRoute = 0x4u;  // NVFP4_DEVICE_BAD_ROUTE

// ---- plan --------------------------------------------------------------------------------

// Every warp owns a run of consecutive slots, every CTA of the cluster consecutive runs. Counts
// per (warp, expert) are summed over the warps, the CTAs' totals are exchanged through
// distributed shared memory, and the exclusive prefix (expert, CTA, warp) is the row of the first
// slot of that expert in that run; a second walk over the run hands the rows out in slot order.
// So the order is that of a stable sort, whatever the timing.
//
// Rows of one expert in one run are consecutive. STAGED: the warp sorts its run in shared memory
// and writes slot_of_row in row order, so that a store instruction touches a few sectors instead
// of 32 scattered ones.

// Expert e's word of a warp's counters: padded so that lanes 8 experts apart meet no bank twice.
__device__ __forceinline__ int plan_word(int e) { return e + (e >> 3); }
constexpr int kPlanWords = kMaxSegments + kMaxSegments / 8;

template <typename Id, bool STAGED>
__global__ void __launch_bounds__(kPlanThreads) moe_plan_kernel(
    const Id* __restrict__ ids, int32_t n, int32_t run, int32_t E, int32_t* row_of_slot,
    int32_t* slot_of_row, int32_t* offsets, uint32_t* status) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t plan_smem[];
  __shared__ uint32_t total[kMaxSegments], base[kPlanWords];
  __shared__ uint32_t scan[kMaxSegments / 32];
  __shared__ uint32_t live;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, warps = threads / 32;
  // per warp and expert: next position in the run's order (STAGED) or next row, and what turns the
  // first into the second
  uint32_t* const all_next = plan_smem;
  uint32_t* const all_shift = plan_smem + warps * kPlanWords;
  uint32_t* const next = all_next + warp * kPlanWords;
  uint32_t* const shift = all_shift + warp * kPlanWords;
  uint32_t* const peers_of = plan_smem + (2 * warps + warp) * kPlanWords;
  uint32_t* const sorted = plan_smem + 3 * warps * kPlanWords + (size_t)warp * run;
  for (int i = tid; i < 3 * warps * kPlanWords; i += threads) plan_smem[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_allow_next();

  const int64_t first = ((int64_t)rank * warps + warp) * run;
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
        atomicAdd(&next[plan_word((int)id[j])], 1u);
      else if (id[j] >= E)
        bad = true;
    }
  }
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(status, kBadRoute);
  __syncthreads();
  if (tid < kMaxSegments) {  // exclusive prefixes of the counts over this CTA's warps
    uint32_t sum = 0;
#pragma unroll 8
    for (int w = 0; w < warps; w++) {
      all_shift[w * kPlanWords + plan_word(tid)] = sum;
      sum += all_next[w * kPlanWords + plan_word(tid)];
    }
    total[tid] = sum;
  }
  cluster.sync();
  uint32_t before = 0, all = 0, incl = 0;
  if (tid < kMaxSegments) {
#pragma unroll
    for (int c = 0; c < kPlanMaxCtas; c++) {
      const uint32_t v = c < ctas ? cluster.map_shared_rank(total, c)[tid] : 0u;
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
  cluster.sync();  // also: every CTA has read the others' totals, so none may have ended
  if (tid < kMaxSegments) {
    for (int w = 0; w < warp; w++) incl += scan[w];
    if (rank == 0 && tid < E) offsets[tid] = (int32_t)incl;
    if (tid == kMaxSegments - 1) live = incl;
    base[plan_word(tid)] = incl - all + before;
  }
  __syncthreads();
  uint32_t placed = 0;  // STAGED: the run's held slots
  if (STAGED) {         // counts -> exclusive prefixes over the experts; shift = row - position
    constexpr int kEach = kMaxSegments / 32;
    uint32_t c[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; i++) {
      c[i] = next[plan_word(lane * kEach + i)];
      sum += c[i];
    }
    uint32_t to = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, to, o);
      if (lane >= o) to += v;
    }
    placed = __shfl_sync(0xFFFFFFFFu, to, 31);
    to -= sum;
#pragma unroll
    for (int i = 0; i < kEach; i++) {
      next[plan_word(lane * kEach + i)] = to;
      shift[plan_word(lane * kEach + i)] += base[plan_word(lane * kEach + i)] - to;
      to += c[i];
    }
  } else {
    for (int e = lane; e < kMaxSegments; e += 32)
      next[plan_word(e)] = shift[plan_word(e)] + base[plan_word(e)];
  }
  __syncwarp();
  // Slots that share an expert find each other through a word of shared memory for the expert, one
  // bit a lane (__match_any_sync takes a step for each distinct expert, and a ballot for each bit
  // of the expert about 75 instructions).
  for (int32_t s0 = begin; s0 < end; s0 += 32 * kPlanBatch) {
    int32_t e[kPlanBatch];
#pragma unroll
    for (int j = 0; j < kPlanBatch; j++) {
      const int32_t s = s0 + 32 * j + lane;
      const Id id = s < end ? ids[s] : (Id)-1;
      e[j] = id >= 0 && id < E ? plan_word((int32_t)id) : -1;
    }
#pragma unroll
    for (int j = 0; j < kPlanBatch; j++) {
      const int32_t s = s0 + 32 * j + lane;
      if (s0 + 32 * j >= end) break;
      if (e[j] >= 0) atomicOr(&peers_of[e[j]], 1u << lane);
      __syncwarp();
      uint32_t peers = 0, at = 0;
      if (e[j] >= 0) {
        peers = peers_of[e[j]];
        at = next[e[j]] + __popc(peers & ((1u << lane) - 1u));
      }
      __syncwarp();
      if (e[j] >= 0 && (peers >> lane) == 1u) {  // the expert's last lane
        next[e[j]] = at + 1;
        peers_of[e[j]] = 0;
      }
      __syncwarp();
      if (s < end) {
        int32_t row = -1;
        if (e[j] >= 0) {
          row = (int32_t)(STAGED ? at + shift[e[j]] : at);
          if (STAGED) sorted[at] = ((uint32_t)(s - begin) << 9) | (uint32_t)e[j];
          else slot_of_row[row] = s;
        }
        row_of_slot[s] = row;
      }
    }
  }
  if (STAGED) {
    __syncwarp();
    for (uint32_t i = lane; i < placed; i += 32) {
      const uint32_t v = sorted[i];
      slot_of_row[i + shift[v & 511u]] = begin + (int32_t)(v >> 9);
    }
  }
  for (int64_t r = (int64_t)live + rank * threads + tid; r < n; r += (int64_t)ctas * threads)
    slot_of_row[r] = -1;
}

// ---- rows of a token ---------------------------------------------------------------------

// A warp owns a token (or a range of its row's vectors): lane i holds the token's i-th held row and
// that slot's choice, in the order of the choices.
struct TokenRows {
  int32_t row, slot;
  int count;
};

__device__ __forceinline__ TokenRows load_token_rows(const int32_t* row_of_slot, int64_t token,
                                                     int32_t K, int64_t P, int2 (*scratch)[32],
                                                     uint32_t* status) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t row = lane < K ? row_of_slot[token * K + lane] : -1;
  if (row >= P) {
    atomicOr(status, kBadRoute);
    row = -1;
  }
  const uint32_t held = __ballot_sync(0xFFFFFFFFu, row >= 0);
  if (row >= 0) scratch[warp][__popc(held & ((1u << lane) - 1u))] = make_int2(row, lane);
  __syncwarp();
  const int2 v = scratch[warp][lane];
  return {v.x, v.y, __popc(held)};
}

__device__ __forceinline__ int64_t live_rows(const int32_t* offsets, int32_t E, int64_t P) {
  const int64_t v = offsets[E - 1];
  return v < 0 ? 0 : (v < P ? v : P);
}

__device__ __forceinline__ uint32_t pack_bf16(uint64_t v) {
  const float2 f = f2_unpack(v);
  const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// ---- dispatch ----------------------------------------------------------------------------

// The expert of a packed row: the first whose end is past it (E when there is none).
__device__ __forceinline__ int expert_of(const int32_t* ends, int32_t E, int32_t row) {
  int lo = 0, hi = E;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > row) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// TW warps per token, neighbouring ones taking neighbouring 32 vectors of its row; a CTA holds its
// warps / TW tokens. The token's maximum is joined in shared memory, so that it costs one atomic
// for each of its experts. ONE: the grid is one cluster, which joins the experts' maxima in its
// first CTA's shared memory and writes all of amax itself, so that a small call needs no clearing
// of amax before it.
constexpr int kCopyMaxWarps = 16;
constexpr int64_t kOneClusterTokens = 8;  // a CTA of 16 warps each
template <int TW, int BATCH, bool ONE>
__global__ void __launch_bounds__(32 * kCopyMaxWarps, 2) moe_dispatch_kernel(
    const uint4* __restrict__ x, const int32_t* __restrict__ row_of_slot,
    const int32_t* __restrict__ offsets, int64_t T, int32_t K, int32_t E, int64_t nv, uint4* packed,
    uint32_t* amax, uint32_t* status) {
  namespace cg = cooperative_groups;
  __shared__ int2 scratch[kCopyMaxWarps][32];
  __shared__ int32_t ends[kMaxSegments];
  __shared__ uint32_t top[kCopyMaxWarps], joint[ONE ? kMaxSegments : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int mine = warp / TW, sub = warp % TW;  // the CTA's token, the warp's part of it
  if (lane == 0) top[warp] = 0u;
  if (ONE)
    for (int e = tid; e < kMaxSegments; e += blockDim.x) joint[e] = 0u;
  pdl_wait();
  pdl_allow_next();
  const int64_t token = (int64_t)blockIdx.x * (blockDim.x / 32 / TW) + mine, P = T * K;
  for (int e = tid; e < E; e += blockDim.x) ends[e] = offsets[e];
  if (ONE) cg::this_cluster().sync();
  else __syncthreads();
  TokenRows rows = {0, 0, 0};
  if (token < T) {
    rows = load_token_rows(row_of_slot, token, K, P, scratch, status);
    uint32_t m = 0;
    for (int64_t at = sub * 32; at < nv; at += 32 * TW * BATCH) {  // every lane: shuffles
      const int64_t v = at + lane;
      uint4 q[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; j++)
        q[j] = v + 32 * TW * j < nv ? __ldg(x + token * nv + v + 32 * TW * j)
                                    : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int j = 0; j < BATCH; j++)
        m = vmax2(m, vmax2(vmax2(abs2(q[j].x), abs2(q[j].y)), vmax2(abs2(q[j].z), abs2(q[j].w))));
      for (int k = 0; k < rows.count; k++) {
        uint4* to = packed + __shfl_sync(0xFFFFFFFFu, rows.row, k) * nv + v;
#pragma unroll
        for (int j = 0; j < BATCH; j++)
          if (v + 32 * TW * j < nv) to[32 * TW * j] = q[j];
      }
    }
    m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
    if (lane == 0 && m != 0u) atomicMax(&top[mine], m);
  }
  __syncthreads();
  if (amax != nullptr && sub == 0 && lane < rows.count) {
    const int e = expert_of(ends, E, rows.row);
    const uint32_t m = top[mine] << 16;
    if (e < E) atomicMax(ONE ? cg::this_cluster().map_shared_rank(joint, 0) + e : amax + e, m);
  }
  if (token < T)
    for (int64_t r = live_rows(ends, E, P) + token; r < P; r += T)
      for (int64_t v = sub * 32 + lane; v < nv; v += 32 * TW)
        packed[r * nv + v] = make_uint4(0u, 0u, 0u, 0u);
  if (ONE) {
    cg::this_cluster().sync();
    if (amax != nullptr && blockIdx.x == 0)
      for (int e = tid; e < E; e += blockDim.x) amax[e] = joint[e];
  }
}

// Short rows, at most kNarrowVecs vectors: a warp per token, CTAs that stay for many tokens and
// join the experts' maxima in shared memory. One atomic a slot into the few lines of amax runs at 2
// per ns: 16384 x 8 slots of 512 columns and 64 experts take 66.0 us that way and 24.9 us this way.
constexpr int kNarrowVecs = 128;
constexpr int kNarrowThreads = 512;
__global__ void __launch_bounds__(kNarrowThreads, 2) moe_dispatch_narrow_kernel(
    const uint4* __restrict__ x, const int32_t* __restrict__ row_of_slot,
    const int32_t* __restrict__ offsets, int64_t T, int32_t K, int32_t E, int64_t nv, uint4* packed,
    uint32_t* amax, uint32_t* status) {
  constexpr int kWarps = kNarrowThreads / 32, kBatch = kNarrowVecs / 32;
  __shared__ int2 scratch[kWarps][32];
  __shared__ int32_t ends[kMaxSegments];
  __shared__ uint32_t joint[kMaxSegments];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t P = T * K;
  pdl_wait();
  pdl_allow_next();
  for (int e = tid; e < E; e += kNarrowThreads) {
    ends[e] = offsets[e];
    joint[e] = 0u;
  }
  __syncthreads();
  const int64_t live = live_rows(ends, E, P);
  for (int64_t token = (int64_t)blockIdx.x * kWarps + warp; token < T;
       token += (int64_t)gridDim.x * kWarps) {
    uint4 q[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; j++)
      q[j] = lane + 32 * j < nv ? __ldg(x + token * nv + lane + 32 * j)
                                : make_uint4(0u, 0u, 0u, 0u);
    const TokenRows rows = load_token_rows(row_of_slot, token, K, P, scratch, status);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kBatch; j++)
      m = vmax2(m, vmax2(vmax2(abs2(q[j].x), abs2(q[j].y)), vmax2(abs2(q[j].z), abs2(q[j].w))));
    for (int k = 0; k < rows.count; k++) {
      uint4* to = packed + __shfl_sync(0xFFFFFFFFu, rows.row, k) * nv + lane;
#pragma unroll
      for (int j = 0; j < kBatch; j++)
        if (lane + 32 * j < nv) to[32 * j] = q[j];
    }
    m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
    if (lane < rows.count) {
      const int e = expert_of(ends, E, rows.row);
      if (e < E) atomicMax(&joint[e], m << 16);
    }
    for (int64_t r = live + token; r < P; r += T)
      for (int64_t v = lane; v < nv; v += 32) packed[r * nv + v] = make_uint4(0u, 0u, 0u, 0u);
    __syncwarp();  // `scratch` has been read
  }
  __syncthreads();
  if (amax != nullptr)
    for (int e = tid; e < E; e += kNarrowThreads)
      if (joint[e]) atomicMax(amax + e, joint[e]);
}

// ---- combine and the gradient of dispatch ------------------------------------------------

// out[t] = sum over the token's held rows of w * y[row], in the order of its choices, in binary32;
// a warp per token and range of its row. A lane has 8 loads in flight: VECS vectors of 8 / VECS
// rows.
template <bool WEIGHTED, int VECS>
__global__ void __launch_bounds__(kRouteThreads) moe_gather_sum_kernel(
    const uint4* __restrict__ y, const float* __restrict__ weights,
    const int32_t* __restrict__ row_of_slot, int64_t T, int32_t K, int64_t nv, int64_t span,
    uint4* out, uint32_t* status) {
  __shared__ int2 scratch[kRouteThreads / 32][32];
  pdl_wait();
  pdl_allow_next();
  const int lane = threadIdx.x & 31;
  const int64_t token = (int64_t)blockIdx.x * (kRouteThreads / 32) + (threadIdx.x >> 5), P = T * K;
  if (token >= T) return;
  const TokenRows rows = load_token_rows(row_of_slot, token, K, P, scratch, status);
  const float weight = WEIGHTED && lane < rows.count ? weights[token * K + rows.slot] : 0.0f;
  const int64_t v0 = (int64_t)blockIdx.y * span, v1 = v0 + span < nv ? v0 + span : nv;
  constexpr int kRows = 8 / VECS;
  for (int64_t at = v0; at < v1; at += 32 * VECS) {  // every lane, for the shuffles
    const int64_t v = at + lane;
    uint64_t acc[VECS][4];
#pragma unroll
    for (int u = 0; u < VECS; u++)
#pragma unroll
      for (int i = 0; i < 4; i++) acc[u][i] = f2_pack(0.0f, 0.0f);
    for (int k0 = 0; k0 < rows.count; k0 += kRows) {
      uint4 q[kRows][VECS];
#pragma unroll
      for (int j = 0; j < kRows; j++) {
        const int32_t row = __shfl_sync(0xFFFFFFFFu, rows.row, k0 + j);
#pragma unroll
        for (int u = 0; u < VECS; u++)
          q[j][u] = k0 + j < rows.count && v + 32 * u < v1 ? __ldg(y + row * nv + v + 32 * u)
                                                           : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < kRows; j++) {
        if (k0 + j < rows.count) {
          const float w = WEIGHTED ? __shfl_sync(0xFFFFFFFFu, weight, k0 + j) : 1.0f;
          const uint64_t w2 = f2_pack(w, w);
#pragma unroll
          for (int u = 0; u < VECS; u++) {
            const uint32_t e[4] = {q[j][u].x, q[j][u].y, q[j][u].z, q[j][u].w};
#pragma unroll
            for (int i = 0; i < 4; i++)
              acc[u][i] = WEIGHTED ? f2_fma(w2, f2_from_bf16x2(e[i]), acc[u][i])
                                   : f2_add(f2_from_bf16x2(e[i]), acc[u][i]);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < VECS; u++)
      if (v + 32 * u < v1)
        out[token * nv + v + 32 * u] =
            make_uint4(pack_bf16(acc[u][0]), pack_bf16(acc[u][1]), pack_bf16(acc[u][2]),
                       pack_bf16(acc[u][3]));
  }
}

// ---- the gradient of combine -------------------------------------------------------------

// grad_y[row] = w * grad[t] and grad_w[t, k] = <grad[t], y[row]>: TW warps per slot, so that the
// product is summed within a warp or two; the slots of a CTA mostly share a token, whose gradient
// row then comes from L1 (a CTA per token with the row in registers took 170 us at 4096 x 8 rows of
// 7168 columns). Slot i also clears row i when it lies past the last expert's end.
constexpr int kSlotThreads = 256;
template <int TW, int BATCH>
__global__ void __launch_bounds__(kSlotThreads) moe_combine_backward_kernel(
    const uint4* __restrict__ grad, const uint4* __restrict__ y, const float* __restrict__ weights,
    const int32_t* __restrict__ row_of_slot, const int32_t* __restrict__ offsets, int64_t T,
    int32_t K, int32_t E, int64_t nv, uint4* grad_y, float* grad_w, uint32_t* status) {
  __shared__ float red[kSlotThreads / 32];
  pdl_wait();
  pdl_allow_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kThreads = 32 * TW;
  const int mine = warp / TW, sub = warp % TW;
  const int64_t P = T * K;
  const int64_t slot = (int64_t)blockIdx.x * (kSlotThreads / kThreads) + mine;
  const int64_t v0 = sub * 32 + lane;
  float dot = 0.0f;
  if (slot < P) {
    const int64_t token = (uint32_t)slot / (uint32_t)K;
    int64_t row = row_of_slot[slot];
    if (row >= P) {
      if (lane == 0) atomicOr(status, kBadRoute);
      row = -1;
    }
    if (row >= 0) {
      const float w = weights[slot];
      const uint64_t w2 = f2_pack(w, w);
      uint64_t s = f2_pack(0.0f, 0.0f);
      const uint4 *g = grad + token * nv, *from = y + row * nv;
      uint4* to = grad_y + row * nv;
      for (int64_t v = v0; v < nv; v += kThreads * BATCH) {
        uint4 a[BATCH], b[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; j++) {
          const bool in = v + kThreads * j < nv;
          b[j] = in ? __ldg(from + v + kThreads * j) : make_uint4(0u, 0u, 0u, 0u);
          a[j] = in ? __ldg(g + v + kThreads * j) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < BATCH; j++) {
          const uint32_t ae[4] = {a[j].x, a[j].y, a[j].z, a[j].w};
          const uint32_t be[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const uint64_t d = f2_from_bf16x2(ae[i]);
            s = f2_fma(d, f2_from_bf16x2(be[i]), s);
            o[i] = pack_bf16(f2_mul(w2, d));
          }
          if (v + kThreads * j < nv) to[v + kThreads * j] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      const float2 f = f2_unpack(s);
      dot = __fadd_rn(f.x, f.y);
    }
    if (slot >= live_rows(offsets, E, P))
      for (int64_t v = v0; v < nv; v += kThreads)
        grad_y[slot * nv + v] = make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
  if (TW > 1) {
    if (lane == 0) red[warp] = dot;
    __syncthreads();
    for (int i = 1; i < TW; i++) dot += red[mine * TW + i];  // (of the first warp's lanes)
  }
  if (lane == 0 && sub == 0 && slot < P) grad_w[slot] = dot;
}

}  // namespace

constexpr int plan_smem_bytes(int warps, int32_t run, bool staged) {
  return 4 * (3 * warps * kPlanWords + (staged ? warps * run : 0));
}

template <typename Id, bool STAGED>
static cudaError_t prepare_plan() {
  const void* f = reinterpret_cast<const void*>(moe_plan_kernel<Id, STAGED>);
  const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              plan_smem_bytes(kPlanThreads / 32, kPlanMaxRun, STAGED));
}

cudaError_t prepare_moe_kernels(int* plan_ctas) {
  cudaError_t e = cudaSuccess, r;
  if ((r = prepare_plan<int32_t, false>()) != cudaSuccess) e = r;
  if ((r = prepare_plan<int32_t, true>()) != cudaSuccess) e = r;
  if ((r = prepare_plan<int64_t, false>()) != cudaSuccess) e = r;
  if ((r = prepare_plan<int64_t, true>()) != cudaSuccess) e = r;
  // a device with fewer SMs in every GPC (a reduced share) does not hold the large cluster
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanMaxCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = plan_smem_bytes(kPlanThreads / 32, kPlanMaxRun, true);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPlanMaxCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  *plan_ctas = kPlanMaxCtas;
  if (cudaOccupancyMaxActiveClusters(&clusters, moe_plan_kernel<int64_t, true>, &cfg) !=
          cudaSuccess ||
      clusters < 1) {
    (void)cudaGetLastError();
    *plan_ctas = kPlanPortableCtas;
  }
  return e;
}

// A launch of one cluster (the grid is the cluster) with programmatic dependent launch.
template <typename... KernelArgs, typename... Args>
static cudaError_t launch_cluster(void (*kernel)(KernelArgs...), int ctas, int threads, size_t smem,
                                  cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
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
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

template <typename Id>
static cudaError_t launch_plan(const void* ids, int32_t n, int32_t E, int32_t* row_of_slot,
                               int32_t* slot_of_row, int32_t* offsets, uint32_t* status,
                               int plan_ctas, cudaStream_t s) {
  // one CTA against the cluster, 256 threads: 4.1 and 4.2 us at 1024 slots, 5.1 and 4.4 at 2048;
  // the cluster with 256 and with 1024 threads: 5.0 and 6.3 us at 16384
  const int threads = n <= 16384 ? kMaxSegments : kPlanThreads;
  const int ctas = n <= 1024 ? 1 : plan_ctas;
  const int warps = threads / 32;
  const int64_t lanes = (int64_t)ctas * threads;
  const int32_t run = (int32_t)((n + lanes - 1) / lanes * 32);
  // sorted in shared memory against scattered stores: 14.1 and 17.3 us at 262144 slots of 64
  // experts (eight slots an expert in a run), 17.7 and 17.3 us with 256 experts (two)
  const bool staged = ctas > 1 && run >= 4 * E && run <= kPlanMaxRun;
  return launch_cluster(staged ? moe_plan_kernel<Id, true> : moe_plan_kernel<Id, false>, ctas,
                        threads, plan_smem_bytes(warps, run, staged), s,
                        static_cast<const Id*>(ids), n, run, E, row_of_slot, slot_of_row, offsets,
                        status);
}

cudaError_t launch_moe_plan(const void* ids, bool wide, int32_t n, int32_t E, int32_t* row_of_slot,
                            int32_t* slot_of_row, int32_t* offsets, uint32_t* status,
                            int plan_ctas, cudaStream_t s) {
  const auto launch = wide ? launch_plan<int64_t> : launch_plan<int32_t>;
  cudaError_t e = plan_ctas > kPlanPortableCtas && setup_fault() == 2
                      ? cudaErrorInvalidValue
                      : launch(ids, n, E, row_of_slot, slot_of_row, offsets, status, plan_ctas, s);
  // The stream's own context may hold fewer SMs than the device (a green context). Its rejection
  // comes before anything is enqueued; a capture records the launch unchecked.
  if (e != cudaSuccess && plan_ctas > kPlanPortableCtas) {
    (void)cudaGetLastError();
    e = launch(ids, n, E, row_of_slot, slot_of_row, offsets, status, kPlanPortableCtas, s);
  }
  return e;
}

// Grid of a warp per token and range of its row: whole rows when the tokens alone give every SM
// about 64 warps, else ranges of at least 32 vectors.
static dim3 token_grid(int64_t tokens, int64_t nv, int sm_count, int64_t* span) {
  const int64_t want = (int64_t)sm_count * 64;
  int64_t ranges = (want + tokens - 1) / tokens;
  const int64_t most = (nv + 31) / 32;
  if (ranges > most) ranges = most;
  *span = ((nv + ranges - 1) / ranges + 31) / 32 * 32;
  constexpr int kTokens = kRouteThreads / 32;
  return dim3((unsigned)((tokens + kTokens - 1) / kTokens), (unsigned)((nv + *span - 1) / *span));
}

bool moe_dispatch_clears_amax(int64_t T) { return T <= kOneClusterTokens; }

template <int TW, int BATCH>
static cudaError_t launch_dispatch(const void* x, const int32_t* row_of_slot,
                                   const int32_t* offsets, int64_t T, int32_t K, int32_t E,
                                   int64_t nv, void* packed, float* amax, uint32_t* status,
                                   cudaStream_t s) {
  constexpr int kWarps = TW < 4 ? 4 : TW;
  constexpr int64_t kTokens = kWarps / TW;
  return launch_pdl(moe_dispatch_kernel<TW, BATCH, false>,
                    dim3((unsigned)((T + kTokens - 1) / kTokens)), dim3(32 * kWarps), 0, s,
                    static_cast<const uint4*>(x), row_of_slot, offsets, T, K, E, nv,
                    static_cast<uint4*>(packed), reinterpret_cast<uint32_t*>(amax), status);
}

cudaError_t launch_moe_dispatch(const void* x, const int32_t* row_of_slot, const int32_t* offsets,
                                int64_t T, int32_t K, int32_t E, int64_t nv, void* packed,
                                float* amax, uint32_t* status, int sm_count, cudaStream_t s) {
  // up to 8 tokens: 4.5 us and one launch, against 4.7 us and two (8 experts each, 7168 columns)
  if (moe_dispatch_clears_amax(T))
    return launch_cluster(moe_dispatch_kernel<16, 2, true>, (int)T, 32 * 16, 0, s,
                          static_cast<const uint4*>(x), row_of_slot, offsets, T, K, E, nv,
                          static_cast<uint4*>(packed), reinterpret_cast<uint32_t*>(amax), status);
  constexpr int64_t kNarrowTokens = kNarrowThreads / 32;
  const int64_t wave = (int64_t)sm_count * 2;
  // short rows this way and the other: 5.1 and 10.4 us at 2000 x 8 rows of 64 vectors, 10.9 and
  // 31.3 at 16384 x 1 of 128, 52.4 and 63.3 at 16384 x 8 of 128 with 256 experts
  if (nv <= kNarrowVecs) {
    const int64_t ctas = (T + kNarrowTokens - 1) / kNarrowTokens;
    return launch_pdl(moe_dispatch_narrow_kernel, dim3((unsigned)(ctas < wave ? ctas : wave)),
                      dim3(kNarrowThreads), 0, s, static_cast<const uint4*>(x), row_of_slot,
                      offsets, T, K, E, nv, static_cast<uint4*>(packed),
                      reinterpret_cast<uint32_t*>(amax), status);
  }
  // a row in one batch of the lanes' vectors, so that each destination row is written in one burst:
  // eight warps of 4 vectors against four of 8, 4096 x 8 rows of 512, 640, 896 and 1024 vectors:
  // 46.4 and 47.3, 57.2 and 58.5, 80.2 and 81.7, 91.7 and 93.5 us; 8192 x 4 rows of 256, 512, 640
  // and 896: 38.3 and 29.6, 57.4 and 51.4, 67.0 and 64.0, 88.4 and 89.2 us
  if (nv > 512)
    return launch_dispatch<8, 4>(x, row_of_slot, offsets, T, K, E, nv, packed, amax, status, s);
  return launch_dispatch<4, 8>(x, row_of_slot, offsets, T, K, E, nv, packed, amax, status, s);
}

template <int VECS>
static cudaError_t launch_gather(const void* y, const float* weights, const int32_t* row_of_slot,
                                 int64_t T, int32_t K, int64_t nv, void* out, uint32_t* status,
                                 int sm_count, cudaStream_t s) {
  int64_t span = 0;
  const dim3 grid = token_grid(T, nv, sm_count, &span);
  return launch_pdl(
      weights ? moe_gather_sum_kernel<true, VECS> : moe_gather_sum_kernel<false, VECS>, grid,
      dim3(kRouteThreads), 0, s, static_cast<const uint4*>(y), weights, row_of_slot, T, K, nv, span,
      static_cast<uint4*>(out), status);
}

cudaError_t launch_moe_gather_sum(const void* y, const float* weights, const int32_t* row_of_slot,
                                  int64_t T, int32_t K, int64_t nv, void* out, uint32_t* status,
                                  int sm_count, cudaStream_t s) {
  // vectors a lane, 1 / 2 / 4: 58.3 / 50.5 / 51.4 us at 8192 x 4 rows of 512 vectors, 80.4 / 77.5 /
  // 80.9 at 4096 x 8 of 896, 22.5 / 14.4 / 13.3 at 16384 x 1 of 128; with few tokens one vector
  // leaves more warps: 8.0 / 8.9 / 13.8 at 300 x 8 of 896
  if (K == 1) return launch_gather<4>(y, weights, row_of_slot, T, K, nv, out, status, sm_count, s);
  if (K <= 4 || T >= (int64_t)sm_count * 24)
    return launch_gather<2>(y, weights, row_of_slot, T, K, nv, out, status, sm_count, s);
  return launch_gather<1>(y, weights, row_of_slot, T, K, nv, out, status, sm_count, s);
}

template <int TW, int BATCH>
static cudaError_t launch_combine_backward(const void* grad, const void* y, const float* weights,
                                           const int32_t* row_of_slot, const int32_t* offsets,
                                           int64_t T, int32_t K, int32_t E, int64_t nv,
                                           void* grad_y, float* grad_w, uint32_t* status,
                                           cudaStream_t s) {
  constexpr int64_t kSlots = kSlotThreads / 32 / TW;
  return launch_pdl(moe_combine_backward_kernel<TW, BATCH>,
                    dim3((unsigned)((T * K + kSlots - 1) / kSlots)), dim3(kSlotThreads), 0, s,
                    static_cast<const uint4*>(grad), static_cast<const uint4*>(y), weights,
                    row_of_slot, offsets, T, K, E, nv, static_cast<uint4*>(grad_y), grad_w, status);
}

cudaError_t launch_moe_combine_backward(const void* grad, const void* y, const float* weights,
                                        const int32_t* row_of_slot, const int32_t* offsets,
                                        int64_t T, int32_t K, int32_t E, int64_t nv, void* grad_y,
                                        float* grad_w, uint32_t* status, int sm_count,
                                        cudaStream_t s) {
  // four warps of 4 vectors per slot when the slots alone do not give every SM 64 warps, else one
  // of one vector: 3.5 and 5.5 us at 64 x 8 rows of 896 vectors, 42.4 and 43.5 at 1000 x 8, 159.1
  // and 147.3 at 4096 x 8 (one warp of 4 vectors: 152.4; more warps in flight beat more loads a
  // warp)
  if (T * K < (int64_t)sm_count * 64 && nv > 128)
    return launch_combine_backward<4, 4>(grad, y, weights, row_of_slot, offsets, T, K, E, nv,
                                         grad_y, grad_w, status, s);
  return launch_combine_backward<1, 1>(grad, y, weights, row_of_slot, offsets, T, K, E, nv, grad_y,
                                       grad_w, status, s);
}

}  // namespace nvfp4
