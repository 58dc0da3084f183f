// Elementwise operators whose inputs are kept in 8 bits for the backward pass: SwiGLU and RMSNorm.
// A kept tensor is E4M3 codes and one E8M0 scale per 32 consecutive elements of a row (the layout
// nvfp4_mx_dequantize reads). The scale is the smallest power of two that keeps the block's largest
// magnitude within 448: unlike the MX conversion of mx_kernel.cu nothing saturates, so every normal
// element is off by at most half an E4M3 step (2^-4 of itself).
//
// The four passes are bound by DRAM, the norms so above 512 columns and their gradient up to
// 8192: at the measured copy rate of 6787 GB/s their bytes, each read or written once, take 94%
// (SwiGLU 32768 x 2048, 83.9 us), 98% (its gradient, 80.3 us), 84% (RMSNorm 8192 x 4096, 29.8 us;
// 93% at 16384 x 8192) and 98% (its gradient with the residual, 16384 x 8192, 141.3 us) of the
// time. What they had to shed for that was instructions (47 an element in the first norm gradient):
// packed binary32 pairs, 32-byte accesses, bulk copies. Outside that range: a row of up to 512
// columns is a warp's, most of whose lanes idle below 512, and a CTA's barrier serves 8 rows (65536
// x 512: 30.4 us forward, 82%, and 36.6 backward, 68%; 131072 x 256: 48.6 and 54.2; 262144 x 128:
// 91.0 and 98.8, 28% and 25%). The gradient beyond 8192 columns decodes every code twice (8192 x
// 16384: 145 us, 69%; 4096 x 32768: 153 us, 65%).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "nvfp4_device.cuh"
#include "aux_internal.h"
#include "nvfp4_internal.h"
#include "tile_ring.h"

namespace nvfp4 {
namespace {

constexpr uint32_t kBadOffsets = 0x1u;  // NVFP4_DEVICE_BAD_OFFSETS

// 16 BF16 values of one row, half a block of 32 (the other half is in the neighbouring lane), by
// one 32-byte load or store: a warp's request is whole 128-byte lines, with one address a lane.
struct Half32 {
  uint32_t w[8];
};
__device__ __forceinline__ Half32 load_half(const void* p) {
  Half32 h;
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(h.w[0]), "=r"(h.w[1]), "=r"(h.w[2]), "=r"(h.w[3]), "=r"(h.w[4]), "=r"(h.w[5]),
                 "=r"(h.w[6]), "=r"(h.w[7])
               : "l"(p));
  return h;
}
__device__ __forceinline__ void store_half(void* p, const uint32_t (&w)[8]) {
  stg256(p, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t pair_bits(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

constexpr uint32_t kRoundsToInf = 0x7F78u;  // BF16 bits of 1.9375 * 2^127

// The scale byte of a block whose largest magnitude has the BF16 bits `top`. With
// a = 2^(E-127) (1 + m/128) that magnitude, a <= 448 * 2^e = 1.75 * 2^(8+e) first holds at
// e = E - 127 - 8 when m <= 96 and one above it otherwise: ((top + 31) >> 7) - 8, at least 0.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const uint32_t biased = (top + 31u) >> 7;
  return biased > 8u ? biased - 8u : 0u;
}
// 2^(127 - scale), exact for every byte that scale_byte gives
__device__ __forceinline__ float inverse_scale(uint32_t scale) {
  return __uint_as_float((254u - scale) << 23);
}

// The rare block with magnitudes from kRoundsToInf up. Infinities and NaN become NaN (E4M3 has no
// infinity), so they reach the gradient, and do not count for the maximum, which is returned.
// Finite magnitudes from 1.9375 * 2^127 up would round to 2^128, outside binary32: they are kept
// as 1.875 * 2^127, so that what is finite stays finite.
__device__ __forceinline__ uint32_t clean_words(uint32_t (&w)[8]) {
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const int sh = 16 * (i & 1);
    const uint32_t h = (w[i >> 1] >> sh) & 0xFFFFu, b = h & 0x7FFFu;
    uint32_t c = h;
    if (b >= 0x7F80u) c = 0x7FC0u;
    else if (b >= kRoundsToInf) c = (h & 0x8000u) | 0x7F70u;
    if (b < 0x7F80u) top = max(top, b);
    w[i >> 1] = (w[i >> 1] & ~(0xFFFFu << sh)) | (c << sh);
  }
  return top;
}

// E4M3 codes of the lane's half of a block of 32 and the block's scale byte, called by both lanes
// of the pair (lane, lane ^ 1) at once. Scaling by a power of two is exact, so each code is rounded
// once.
__device__ __forceinline__ void keep_half(const Half32& half, uint32_t (&codes)[4],
                                          uint32_t& scale) {
  const uint32_t pair = 3u << (threadIdx.x & 30);
  uint32_t m = abs2(half.w[0]);
#pragma unroll
  for (int i = 1; i < 8; i++) m = vmax2(m, abs2(half.w[i]));
  uint32_t top = pair_bits(m);
  top = max(top, __shfl_xor_sync(pair, top, 1));
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; i++) w[i] = half.w[i];
  if (top >= kRoundsToInf) {  // both lanes of the block
    top = clean_words(w);
    top = max(top, __shfl_xor_sync(pair, top, 1));
  }
  scale = scale_byte(top);
  const float inv = inverse_scale(scale);
  const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float2 lo = f2_unpack(f2_mul(f2_from_bf16x2(w[2 * i]), inv2));
    const float2 hi = f2_unpack(f2_mul(f2_from_bf16x2(w[2 * i + 1]), inv2));
    codes[i] = e4m3x2(lo.x, lo.y) | (e4m3x2(hi.x, hi.y) << 16);
  }
}

// The binary32 value of a scale byte (255 is NaN).
__device__ __forceinline__ float e8m0_value(uint32_t s) {
  return s == 0u ? __uint_as_float(0x00400000u)
                 : (s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s << 23));
}

// 16 codes times a factor, as packed pairs. The factor is the block's scale, alone or times another
// number: E4M3 values times a power of two are exact, so the product is rounded once.
__device__ __forceinline__ void kept_values(const uint4& codes, float factor, uint64_t (&v)[8]) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  const uint64_t f2 = f2_pack(factor, factor);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float2 f = e4m3x2_to_float2((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
    v[i] = f2_mul(f2_pack(f.x, f.y), f2);
  }
}
__device__ __forceinline__ void unpack16(const Half32& h, uint64_t (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = f2_from_bf16x2(h.w[i]);
}
__device__ __forceinline__ uint32_t pack_bf16(uint64_t v) {
  const float2 f = f2_unpack(v);
  return pack_bf16(f.x, f.y);
}

// sigmoid(a) from t = exp(-|a|), which cannot overflow. t is the square of 2^(-|a| log2(e) / 2):
// the approximate instruction flushes subnormal results, which that square root only reaches where
// t itself is below binary32's smallest subnormal.
__device__ __forceinline__ float sigmoid(float a) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(fabsf(a), -0.72134752f)));
  const float t = __fmul_rn(e, e);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, t)));
  return a >= 0.0f ? r : __fmul_rn(t, r);
}

// ---- SwiGLU ------------------------------------------------------------------------------

constexpr int kGluThreads = 256;

// The consecutive items (row, 16 columns) [first, last) of this CTA, a thread every kGluThreads-th.
struct GluWalk {
  int64_t left;      // items the thread still has
  int64_t row;
  int64_t col;       // in items of 16 columns
  int64_t step_row, step_col, per_row;
  __device__ GluWalk(int64_t rows, int64_t per_row_, int64_t per_cta) : per_row(per_row_) {
    const int64_t items = rows * per_row;
    const int64_t first = (int64_t)blockIdx.x * per_cta + threadIdx.x;
    const int64_t last = min(items, ((int64_t)blockIdx.x + 1) * per_cta);
    left = first < last ? (last - first + kGluThreads - 1) / kGluThreads : 0;
    row = first / per_row;
    col = first - row * per_row;
    step_row = kGluThreads / per_row;
    step_col = kGluThreads - step_row * per_row;
  }
  __device__ void next() {
    left--;
    row += step_row;
    col += step_col;
    if (col >= per_row) {
      col -= per_row;
      row++;
    }
  }
};

// Rows before the last expert's end, within [0, M]; an end outside that range is flagged.
__device__ __forceinline__ int64_t live_of(const int32_t* offsets, int32_t E, int64_t M,
                                           uint32_t* status) {
  if (offsets == nullptr) return M;
  const int64_t v = offsets[E - 1];
  if ((v < 0 || v > M) && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, kBadOffsets);
  return v < 0 ? 0 : (v < M ? v : M);
}
// Whether an expert's end lies before the previous one's (the first one's: before 0).
__device__ __forceinline__ bool descends(const int32_t* offsets, int e) {
  return offsets[e] < (e > 0 ? offsets[e - 1] : 0);
}

__global__ void __launch_bounds__(kGluThreads) swiglu_checkpoint_kernel(
    const uint4* __restrict__ h, int64_t M, int64_t F, const int32_t* __restrict__ offsets,
    int32_t E, int64_t per_cta, uint4* y, uint4* codes, uint8_t* scales, uint32_t* amax,
    uint32_t* status) {
  __shared__ int32_t ends[kMaxSegments];
  __shared__ uint32_t top[kMaxSegments];
  pdl_wait();
  pdl_allow_next();
  const int tid = threadIdx.x;
  const int64_t live = live_of(offsets, E, M, status);
  for (int e = tid; e < E; e += kGluThreads) {
    ends[e] = offsets ? offsets[e] : (int32_t)M;
    top[e] = 0u;
    if (blockIdx.x == 0 && offsets && descends(offsets, e)) atomicOr(status, kBadOffsets);
  }
  __syncthreads();
  const int64_t nc = F / 16;
  GluWalk it(M, nc, per_cta);
  int expert = 0;  // of the thread's current row: the first whose end is past it, at most E - 1
  for (int hi = E - 1; expert < hi;) {
    const int mid = (expert + hi) >> 1;
    if (ends[mid] > it.row) hi = mid; else expert = mid + 1;
  }
  uint32_t m = 0u;
  for (; it.left > 0; it.next()) {
    const int64_t r = it.row, c = it.col;
    uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, kg[4] = {0u, 0u, 0u, 0u},
             ku[4] = {0u, 0u, 0u, 0u}, sg = 0u, su = 0u;
    if (r < live) {
      const Half32 g = load_half(h + (r * 2 * nc + c) * 2);
      const Half32 u = load_half(h + (r * 2 * nc + nc + c) * 2);
      while (expert < E - 1 && r >= ends[expert]) {
        if (m) atomicMax(&top[expert], m);
        m = 0u;
        expert++;
      }
      uint32_t mm = 0u;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float a0 = bf16_lo(g.w[i]), a1 = bf16_hi(g.w[i]);
        o[i] = pack_bf16(__fmul_rn(__fmul_rn(a0, sigmoid(a0)), bf16_lo(u.w[i])),
                         __fmul_rn(__fmul_rn(a1, sigmoid(a1)), bf16_hi(u.w[i])));
        mm = vmax2(mm, abs2(o[i]));
      }
      m = max(m, pair_bits(mm));
      keep_half(g, kg, sg);
      keep_half(u, ku, su);
    }
    store_half(y + (r * nc + c) * 2, o);
    codes[r * 2 * nc + c] = make_uint4(kg[0], kg[1], kg[2], kg[3]);
    codes[r * 2 * nc + nc + c] = make_uint4(ku[0], ku[1], ku[2], ku[3]);
    if ((c & 1) == 0) {
      scales[r * nc + c / 2] = (uint8_t)sg;
      scales[r * nc + nc / 2 + c / 2] = (uint8_t)su;
    }
  }
  if (m) atomicMax(&top[expert], m);
  __syncthreads();
  if (amax != nullptr)
    for (int e = tid; e < E; e += kGluThreads)
      if (top[e]) atomicMax(amax + e, top[e] << 16);
}

// dg = dy u s (1 + g (1 - s)), du = dy g s with s = sigmoid(g), from the kept g and u.
__global__ void __launch_bounds__(kGluThreads) swiglu_checkpoint_backward_kernel(
    const uint4* __restrict__ grad, const uint4* __restrict__ codes,
    const uint8_t* __restrict__ scales, int64_t M, int64_t F, const int32_t* __restrict__ offsets,
    int32_t E, int64_t per_cta, uint4* grad_h, uint32_t* status) {
  pdl_wait();
  pdl_allow_next();
  const int64_t live = live_of(offsets, E, M, status);
  if (blockIdx.x == 0 && offsets)
    for (int e = threadIdx.x; e < E; e += kGluThreads)
      if (descends(offsets, e)) atomicOr(status, kBadOffsets);
  const int64_t nc = F / 16;
  for (GluWalk it(M, nc, per_cta); it.left > 0; it.next()) {
    const int64_t r = it.row, c = it.col;
    uint32_t og[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, ou[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (r < live) {
      uint64_t g[8], u[8];
      const Half32 d = load_half(grad + (r * nc + c) * 2);
      const uint4 kg = __ldg(codes + r * 2 * nc + c), ku = __ldg(codes + r * 2 * nc + nc + c);
      kept_values(kg, e8m0_value(scales[r * nc + c / 2]), g);
      kept_values(ku, e8m0_value(scales[r * nc + nc / 2 + c / 2]), u);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float dg[2], du[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const float dy = j ? bf16_hi(d.w[i]) : bf16_lo(d.w[i]);
          const float2 av = f2_unpack(g[i]), bv = f2_unpack(u[i]);
          const float a = j ? av.y : av.x, b = j ? bv.y : bv.x;
          const float s = sigmoid(a);
          const float slope = __fmul_rn(s, __fmaf_rn(a, __fsub_rn(1.0f, s), 1.0f));
          dg[j] = __fmul_rn(__fmul_rn(dy, b), slope);
          du[j] = __fmul_rn(dy, __fmul_rn(a, s));
        }
        og[i] = pack_bf16(dg[0], dg[1]);
        ou[i] = pack_bf16(du[0], du[1]);
      }
    }
    store_half(grad_h + (r * 2 * nc + c) * 2, og);
    store_half(grad_h + (r * 2 * nc + nc + c) * 2, ou);
  }
}

// ---- RMSNorm -----------------------------------------------------------------------------

// A group of `wpr` warps owns a row, ITEMS x 16 columns a thread; a CTA of at most WARPS warps
// works on tiles of `groups` consecutive rows. A tile is contiguous in memory: one thread fetches
// it by bulk copies into a ring of STAGES tiles in shared memory, ahead of the tile that is summed,
// so that neither the loads nor their addresses cost the other threads instructions, and DRAM stays
// busy across the barrier of the sum. Where registers and shared memory leave room, several CTAs
// share an SM, one computing while another waits at its barrier: forward 3, 2, 1 and 1 by width
// (RmsForward0 to 3), backward 2, 1, 1 and 1.
constexpr int kMaxJointN = 2048;  // a CTA with more than one group has rows up to this
constexpr uint64_t kTileWaitNs = 2000000000ull;
constexpr uint32_t kTimeout = 0x2u;  // NVFP4_DEVICE_TIMEOUT

struct RmsShape {
  int wpr, groups;
};
RmsShape rms_shape(int64_t N, int warps, int items) {
  RmsShape s;
  const int64_t per_warp = 512 * items;
  s.wpr = (int)((N + per_warp - 1) / per_warp);
  s.groups = warps / s.wpr;
  return s;
}

// A thread's waits for the CTA's tiles (thread 0 is the ring's owner). A wait that gives up is
// reported.
template <int STAGES>
struct TileWaits : TileRing<STAGES> {
  uint64_t* full;
  uint32_t* status;
  __device__ TileWaits(uint64_t* full_, uint32_t* status_) : full(full_), status(status_) {}
  // `first` is the tile's first row; the next tiles start `step` rows on, below M.
  __device__ void wait(int64_t first, int64_t step, int64_t M) {
    TileRing<STAGES>::wait(
        threadIdx.x == 0,
        [&](int stage, uint32_t parity) {
          if (mbar_wait_bounded(&full[stage], parity, kTileWaitNs)) return true;
          atomicOr(status, kTimeout);
          return false;
        },
        [&](int i) { return first + i * step < M; });
  }
};

// Sum over each group's threads: shuffles, then the warps' sums through shared memory, in an order
// that does not depend on time; `red` has two halves used in turn. The barrier is the CTA's, so
// that after it every thread has left the previous tile.
template <int WARPS>
__device__ __forceinline__ float group_sum(uint64_t pair, float (*red)[WARPS], int turn, int group,
                                           int wpr) {
  const float2 f = f2_unpack(pair);
  float s = __fadd_rn(f.x, f.y);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[turn][threadIdx.x >> 5] = s;
  __syncthreads();
  if (wpr == 1) return s;
  s = lane < wpr ? red[turn][group * wpr + lane] : 0.0f;
#pragma unroll
  for (int o = WARPS / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return __shfl_sync(0xFFFFFFFFu, s, 0);
}

// w + bias of 16 columns as packed pairs
__device__ __forceinline__ void biased_weight(const Half32& weight, float bias, uint64_t (&w)[8]) {
  unpack16(weight, w);
  const uint64_t b2 = f2_pack(bias, bias);
#pragma unroll
  for (int i = 0; i < 8; i++) w[i] = f2_add(w[i], b2);
}

// Keeps the packed words in registers, not their widened values, from the sum to the output.
template <int ITEMS>
__device__ __forceinline__ void hold_packed(Half32 (&h)[ITEMS]) {
#pragma unroll
  for (int j = 0; j < ITEMS; j++)
#pragma unroll
    for (int i = 0; i < 8; i++) asm volatile("" : "+r"(h[j].w[i]));
}

__device__ __forceinline__ Half32 shared_half(const uint8_t* at) {
  const uint4* p = reinterpret_cast<const uint4*>(at);
  const uint4 a = p[0], b = p[1];
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// WARPS warps a CTA, ITEMS x 16 columns a thread, STAGES tiles in the ring, CTAS CTAs an SM.
template <int WARPS, int ITEMS, int STAGES, int CTAS>
__global__ void __launch_bounds__(32 * WARPS, CTAS) rmsnorm_checkpoint_kernel(
    const uint4* __restrict__ x, const uint4* __restrict__ weight, int64_t M, int32_t N, float eps,
    float bias, int wpr, int groups, uint4* y, uint4* codes, uint8_t* scales, float* rstd,
    uint32_t* amax, uint32_t* status) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[STAGES];
  __shared__ float red[2][WARPS];
  __shared__ uint32_t top[WARPS];
  constexpr int kStage = WARPS * 32 * ITEMS * 32;  // bytes
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = warp / wpr, at = tid - group * wpr * 32, threads = wpr * 32;
  const int nc = N / 16;
  const float inv_n = 1.0f / (float)N;
  if (tid == 0) {
    for (int i = 0; i < STAGES; i++) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_allow_next();
  const int64_t step = (int64_t)gridDim.x * groups;
  auto fetch = [&](int stage, int64_t row) {  // thread 0
    if (row >= M) return;
    const int64_t rows = M - row < groups ? M - row : groups;
    const uint32_t bytes = (uint32_t)(rows * N * 2);
    mbar_expect_tx(&full[stage], bytes);
    bulk_load(ring + stage * kStage, x + row * nc * 2, bytes, &full[stage]);
  };
  int64_t first = (int64_t)blockIdx.x * groups;  // of the tile
  if (tid == 0)
    for (int i = 0; i < TileRing<STAGES>::kAhead; i++) fetch(i, first + i * step);
  TileWaits<STAGES> tiles(full, status);
  uint32_t m = 0u;
  int turn = 0;
  const uint8_t* const mine = ring + ((size_t)group * nc + at) * 32;
  for (; first < M; first += step) {
    const int64_t r = first + group, pos = r * nc + at;
    const bool live = r < M;
    tiles.wait(first, step, M);
    Half32 w[ITEMS];
    uint64_t s = f2_pack(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      if (!live || at + j * threads >= nc) break;
      w[j] = shared_half(mine + tiles.stage * kStage + j * threads * 32);
      uint64_t v[8];
      unpack16(w[j], v);
#pragma unroll
      for (int i = 0; i < 8; i++) s = f2_fma(v[i], v[i], s);
    }
    const float sum = group_sum<WARPS>(s, red, turn, group, wpr);
    // every thread has read this tile into registers: its stage and all before it are free
    if (tid == 0 && !tiles.dead)
      fetch(tiles.stage == 0 ? STAGES - 1 : tiles.stage - 1, first + (STAGES - 1) * step);
    tiles.next();
    turn ^= 1;
    if (!live) continue;
    hold_packed(w);
    const float rs = rsqrtf(__fmaf_rn(sum, inv_n, eps));
    const uint64_t rs2 = f2_pack(rs, rs);
    if (at == 0) rstd[r] = rs;
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int c = at + j * threads;
      if (c >= nc) break;
      const int64_t p = pos + j * threads;
      uint64_t v[8], g[8];
      uint32_t o[8], k[4], sc;
      unpack16(w[j], v);
      biased_weight(load_half(weight + 2 * c), bias, g);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        o[i] = pack_bf16(f2_mul(g[i], f2_mul(v[i], rs2)));
        m = vmax2(m, abs2(o[i]));
      }
      store_half(y + 2 * p, o);
      keep_half(w[j], k, sc);
      codes[p] = make_uint4(k[0], k[1], k[2], k[3]);
      if ((c & 1) == 0) scales[p / 2] = (uint8_t)sc;  // (rows are an even number of halves)
    }
  }
  m = __reduce_max_sync(0xFFFFFFFFu, pair_bits(m));
  if (lane == 0) top[warp] = m;
  __syncthreads();
  if (warp == 0) {
    m = __reduce_max_sync(0xFFFFFFFFu, lane < (int)(blockDim.x >> 5) ? top[lane] : 0u);
    if (lane == 0) atomicMax(amax, m << 16);
  }
}

// With xh = x * rstd and g = (w + bias) dy: dx = rstd (g - xh mean(g xh)) [+ residual], and
// dw = sum over rows of dy xh. A thread keeps its columns' share of dw over all of its rows; the
// groups of a CTA are added in shared memory in order and each CTA writes one row of `partial`, so
// that the sum's order depends on the grid alone.
__host__ __device__ constexpr int rms_column_bytes(bool res) { return res ? 5 : 3; }

template <int WARPS, int ITEMS, int STAGES, int CTAS, bool RES>
__global__ void __launch_bounds__(32 * WARPS, CTAS) rmsnorm_checkpoint_backward_kernel(
    const uint4* __restrict__ grad, const uint4* __restrict__ codes,
    const uint8_t* __restrict__ scales, const float* __restrict__ rstd,
    const uint4* __restrict__ weight, int64_t M, int32_t N, float bias, int wpr, int groups,
    const uint4* __restrict__ residual, uint4* grad_x, float* partial, uint32_t* status) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[STAGES];
  __shared__ float red[2][WARPS];
  __shared__ float4 cols[kMaxJointN / 4];  // the groups' joint sums
  constexpr int kColumns = WARPS * 32 * ITEMS * 16;
  constexpr int kStage = kColumns * rms_column_bytes(RES);  // grad, residual, codes
  constexpr int kCodes = kColumns * (RES ? 4 : 2);
  const int tid = threadIdx.x, warp = tid >> 5;
  const int group = warp / wpr, at = tid - group * wpr * 32, threads = wpr * 32;
  const int nc = N / 16;
  const float inv_n = 1.0f / (float)N;
  if (tid == 0) {
    for (int i = 0; i < STAGES; i++) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_allow_next();
  constexpr bool kHold = ITEMS == 1;  // xh and g stay in registers from the sum to the output
  uint64_t dw[ITEMS][8], w[8], h[8], g[8];
#pragma unroll
  for (int j = 0; j < ITEMS; j++)
#pragma unroll
    for (int i = 0; i < 8; i++) dw[j][i] = f2_pack(0.0f, 0.0f);
  if (ITEMS == 1 && at < nc) biased_weight(load_half(weight + 2 * at), bias, w);
  const int64_t step = (int64_t)gridDim.x * groups;
  auto fetch = [&](int stage, int64_t row) {  // thread 0
    if (row >= M) return;
    const int64_t rows = M - row < groups ? M - row : groups;
    const uint32_t n = (uint32_t)(rows * N);
    uint8_t* to = ring + stage * kStage;
    mbar_expect_tx(&full[stage], n * rms_column_bytes(RES));
    bulk_load(to, grad + row * nc * 2, 2 * n, &full[stage]);
    bulk_load(to + kCodes, codes + row * nc, n, &full[stage]);
    if (RES) bulk_load(to + kColumns * 2, residual + row * nc * 2, 2 * n, &full[stage]);
  };
  // the scale bytes and the row's rstd come one tile ahead, in registers
  uint32_t next_sc[ITEMS];
  float next_rs = 0.0f;
  auto fetch_scales = [&](int64_t row) {
    if (row < M) {
      next_rs = __ldg(rstd + row);
#pragma unroll
      for (int j = 0; j < ITEMS; j++) {
        const int c = at + j * threads;
        if (c < nc) next_sc[j] = __ldg(scales + (row * nc + c) / 2);
      }
    }
  };
  int64_t first = (int64_t)blockIdx.x * groups;  // of the tile
  if (tid == 0)
    for (int i = 0; i < TileRing<STAGES>::kAhead; i++) fetch(i, first + i * step);
  fetch_scales(first + group);
  TileWaits<STAGES> tiles(full, status);
  int turn = 0;
  const uint8_t* const mine = ring + ((size_t)group * nc + at) * 32;
  const uint8_t* const mine8 = ring + kCodes + ((size_t)group * nc + at) * 16;
  for (; first < M; first += step) {
    const int64_t r = first + group;
    const bool live = r < M;
    const float rs = next_rs;
    float factor[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; j++) factor[j] = __fmul_rn(e8m0_value(next_sc[j]), rs);
    fetch_scales(r + step);
    tiles.wait(first, step, M);
    const int at_stage = tiles.stage * kStage;
    auto prepare = [&](int j, uint64_t (&d)[8]) {  // dy, xh and g of the thread's j-th columns
      const uint4 k = *reinterpret_cast<const uint4*>(mine8 + at_stage + j * threads * 16);
      kept_values(k, factor[j], h);
      unpack16(shared_half(mine + at_stage + j * threads * 32), d);
      if (ITEMS > 1) biased_weight(load_half(weight + 2 * (at + j * threads)), bias, w);
#pragma unroll
      for (int i = 0; i < 8; i++) g[i] = f2_mul(w[i], d[i]);
    };
    uint64_t s = f2_pack(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int c = at + j * threads;
      if (!live || c >= nc) break;
      uint64_t d[8];
      prepare(j, d);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        dw[j][i] = f2_fma(d[i], h[i], dw[j][i]);
        s = f2_fma(g[i], h[i], s);
      }
    }
    const float mean = __fmul_rn(group_sum<WARPS>(s, red, turn, group, wpr), inv_n);
    turn ^= 1;
    // every thread has left the previous tile: its stage takes the tile STAGES - 1 ahead
    if (STAGES > 1 && tid == 0 && !tiles.dead)
      fetch(tiles.stage == 0 ? STAGES - 1 : tiles.stage - 1, first + (STAGES - 1) * step);
    tiles.next();
    const uint64_t rs2 = f2_pack(rs, rs), minus = f2_pack(-mean, -mean);
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int c = at + j * threads;
      if (!live || c >= nc) break;
      uint64_t d[8], e[8];
      uint32_t o[8];
      if (!kHold) prepare(j, d);
      if (RES) unpack16(shared_half(mine + at_stage + kColumns * 2 + j * threads * 32), e);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const uint64_t q = f2_fma(h[i], minus, g[i]);
        o[i] = pack_bf16(RES ? f2_fma(rs2, q, e[i]) : f2_mul(rs2, q));
      }
      store_half(grad_x + 2 * (r * nc + c), o);
    }
    if (STAGES == 1) {
      __syncthreads();
      if (tid == 0 && !tiles.dead) fetch(0, first + step);
    }
  }
  float4* out = reinterpret_cast<float4*>(partial + (int64_t)blockIdx.x * N);
  for (int g = 0; g < groups; g++) {
    if (group == g) {
#pragma unroll
      for (int j = 0; j < ITEMS; j++) {
        const int c = at + j * threads;
        if (c >= nc) break;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float2 lo = f2_unpack(dw[j][2 * i]), hi = f2_unpack(dw[j][2 * i + 1]);
          float4 v = make_float4(lo.x, lo.y, hi.x, hi.y);
          if (g > 0) {
            const float4 p = cols[c * 4 + i];
            v = make_float4(p.x + v.x, p.y + v.y, p.z + v.z, p.w + v.w);
          }
          if (g == groups - 1) out[c * 4 + i] = v;
          else cols[c * 4 + i] = v;
        }
      }
    }
    if (groups > 1) __syncthreads();
  }
}

// grad_weight[n] = sum of the `parts` rows of partial [parts][N]: 32 columns a CTA, eight warps
// over the rows, added in a fixed order.
constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(32 * kSumWarps) column_sum_kernel(
    const float* __restrict__ partial, int parts, int64_t N, float* out) {
  __shared__ float red[kSumWarps][32];
  pdl_wait();
  pdl_allow_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
#pragma unroll 4
  for (int p = warp; p < parts; p += kSumWarps) s += partial[p * N + n];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    for (int i = 1; i < kSumWarps; i++) s += red[i][lane];
    out[n] = s;
  }
}

// Items of a CTA: about eight CTAs an SM, and at most four items a thread, so that the resident
// CTAs sweep the tensors in address order: one long range for each of eight CTAs an SM took 97.6 us
// instead of 86.3 forward and 83.2 instead of 80.3 backward at 32768 x 2048.
int64_t glu_per_cta(int64_t items, int sm_count, int* grid) {
  const int64_t most = (int64_t)sm_count * 8;
  int64_t per = (items + most - 1) / most;
  if (per > 4 * kGluThreads) per = 4 * kGluThreads;
  if (per < items / (1 << 30)) per = items / (1 << 30);  // the grid stays within 31 bits
  per = (per + kGluThreads - 1) / kGluThreads * kGluThreads;
  *grid = (int)((items + per - 1) / per);
  return per;
}

int rms_grid(const RmsShape& f, int64_t M, int64_t wave) {
  const int64_t ctas = (M + f.groups - 1) / f.groups;
  return (int)(ctas < wave ? ctas : wave);
}

// One kernel's shape, as template arguments of both directions.
template <int WARPS, int ITEMS, int STAGES, int CTAS>
struct RmsForward {
  static constexpr int kSmem = STAGES * WARPS * 32 * ITEMS * 32;
  static cudaError_t prepare() {
    return cudaFuncSetAttribute(rmsnorm_checkpoint_kernel<WARPS, ITEMS, STAGES, CTAS>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  }
  static cudaError_t launch(const RmsArgs& a, int sm_count, cudaStream_t s) {
    const RmsShape f = rms_shape(a.N, WARPS, ITEMS);
    return launch_pdl(rmsnorm_checkpoint_kernel<WARPS, ITEMS, STAGES, CTAS>,
                      dim3(rms_grid(f, a.M, (int64_t)sm_count * CTAS)),
                      dim3(f.wpr * f.groups * 32), kSmem, s, static_cast<const uint4*>(a.x),
                      static_cast<const uint4*>(a.weight), a.M, (int32_t)a.N, a.eps, a.bias, f.wpr,
                      f.groups, static_cast<uint4*>(a.y), static_cast<uint4*>(a.codes), a.scales,
                      a.rstd, reinterpret_cast<uint32_t*>(a.amax), a.status);
  }
};

template <int WARPS, int ITEMS, int STAGES, int CTAS, bool RES>
struct RmsBackward {
  static constexpr int kSmem = STAGES * WARPS * 32 * ITEMS * 16 * rms_column_bytes(RES);
  static cudaError_t prepare() {
    return cudaFuncSetAttribute(rmsnorm_checkpoint_backward_kernel<WARPS, ITEMS, STAGES, CTAS, RES>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  }
  static cudaError_t launch(const RmsArgs& a, int sm_count, cudaStream_t s) {
    const RmsShape f = rms_shape(a.N, WARPS, ITEMS);
    int64_t wave = (int64_t)sm_count * CTAS;
    if (wave > kRmsMaxPartials) wave = kRmsMaxPartials;
    const int grid = rms_grid(f, a.M, wave);
    const cudaError_t e = launch_pdl(
        rmsnorm_checkpoint_backward_kernel<WARPS, ITEMS, STAGES, CTAS, RES>, dim3(grid),
        dim3(f.wpr * f.groups * 32), kSmem, s, static_cast<const uint4*>(a.grad),
        static_cast<const uint4*>(a.codes), a.scales, a.rstd, static_cast<const uint4*>(a.weight),
        a.M, (int32_t)a.N, a.bias, f.wpr, f.groups, static_cast<const uint4*>(a.residual),
        static_cast<uint4*>(a.grad_x), a.partial, a.status);
    if (e != cudaSuccess) return e;
    return launch_pdl(column_sum_kernel, dim3((unsigned)(a.N / 32)), dim3(32 * kSumWarps), 0, s,
                      a.partial, grid, a.N, a.grad_weight);
  }
};

// By the row's columns: up to 4096, 8192, 16384, 32768. Forward, 8192 x 4096: 29.7 us with three
// CTAs of 8 warps an SM, 31.0 with two of 16; 16384 x 8192: 112.5 with two of 8 warps and 32
// columns a thread, 106.5 with two of 16 warps and 16. Backward, 16384 x 8192 with the residual:
// 158.7 with two of 8 warps and 32 columns a thread (which decode every code twice), 141.3 with one
// of 16 warps and 16; 32768 x 4096: 115.6 with two of 8 warps, 117.4 with one of 16. Beyond 8192
// columns xh and g are not kept from the sum to the output beside the weight gradient's
// accumulators (kept together they took longer; xh alone was not tried), so the codes are decoded
// twice. The weights are read for every row, so the ring must leave them L1: 8192 x 16384 takes 145
// us with two stages and 167 with four (with the residual 170 us, 82%). 4096 x 32768: 153 us with
// two stages, 162 with one; with the residual one is all that fits, and no load overlaps the
// computation (211 us, 66%).
using RmsForward0 = RmsForward<8, 1, 4, 3>;
using RmsForward1 = RmsForward<16, 1, 4, 2>;
using RmsForward2 = RmsForward<16, 2, 4, 1>;
using RmsForward3 = RmsForward<16, 4, 3, 1>;
template <bool RES> using RmsBackward0 = RmsBackward<8, 1, 4, 2, RES>;
template <bool RES> using RmsBackward1 = RmsBackward<16, 1, 4, 1, RES>;
template <bool RES> using RmsBackward2 = RmsBackward<16, 2, 2, 1, RES>;
template <bool RES> using RmsBackward3 = RmsBackward<16, 4, RES ? 1 : 2, 1, RES>;

template <bool RES>
cudaError_t rms_backward(const RmsArgs& a, int sm_count, cudaStream_t s) {
  if (a.N <= 4096) return RmsBackward0<RES>::launch(a, sm_count, s);
  if (a.N <= 8192) return RmsBackward1<RES>::launch(a, sm_count, s);
  if (a.N <= 16384) return RmsBackward2<RES>::launch(a, sm_count, s);
  return RmsBackward3<RES>::launch(a, sm_count, s);
}

}  // namespace

cudaError_t launch_swiglu_checkpoint(const void* h, int64_t M, int64_t F, const int32_t* offsets,
                                     int32_t E, void* y, void* codes, uint8_t* scales, float* amax,
                                     uint32_t* status, int sm_count, cudaStream_t s) {
  int grid = 0;
  const int64_t per = glu_per_cta(M * (F / 16), sm_count, &grid);
  return launch_pdl(swiglu_checkpoint_kernel, dim3(grid), dim3(kGluThreads), 0, s,
                    static_cast<const uint4*>(h), M, F, offsets, E, per, static_cast<uint4*>(y),
                    static_cast<uint4*>(codes), scales, reinterpret_cast<uint32_t*>(amax), status);
}

cudaError_t launch_swiglu_checkpoint_backward(const void* grad, const void* codes,
                                              const uint8_t* scales, int64_t M, int64_t F,
                                              const int32_t* offsets, int32_t E, void* grad_h,
                                              uint32_t* status, int sm_count, cudaStream_t s) {
  int grid = 0;
  const int64_t per = glu_per_cta(M * (F / 16), sm_count, &grid);
  return launch_pdl(swiglu_checkpoint_backward_kernel, dim3(grid), dim3(kGluThreads), 0, s,
                    static_cast<const uint4*>(grad), static_cast<const uint4*>(codes), scales, M,
                    F, offsets, E, per, static_cast<uint4*>(grad_h), status);
}

cudaError_t prepare_checkpoint_kernels() {
  cudaError_t e = cudaSuccess;
  for (const cudaError_t r :
       {RmsForward0::prepare(), RmsForward1::prepare(), RmsForward2::prepare(),
        RmsForward3::prepare(), RmsBackward0<false>::prepare(), RmsBackward0<true>::prepare(),
        RmsBackward1<false>::prepare(), RmsBackward1<true>::prepare(),
        RmsBackward2<false>::prepare(), RmsBackward2<true>::prepare(),
        RmsBackward3<false>::prepare(), RmsBackward3<true>::prepare()})
    if (r != cudaSuccess) e = r;
  return e;
}

cudaError_t launch_rmsnorm_checkpoint(const RmsArgs& a, int sm_count, cudaStream_t s) {
  if (a.N <= 4096) return RmsForward0::launch(a, sm_count, s);
  if (a.N <= 8192) return RmsForward1::launch(a, sm_count, s);
  if (a.N <= 16384) return RmsForward2::launch(a, sm_count, s);
  return RmsForward3::launch(a, sm_count, s);
}

cudaError_t launch_rmsnorm_checkpoint_backward(const RmsArgs& a, int sm_count, cudaStream_t s) {
  return a.residual ? rms_backward<true>(a, sm_count, s) : rms_backward<false>(a, sm_count, s);
}

}  // namespace nvfp4
