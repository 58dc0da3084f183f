// Elementwise operators whose inputs are kept in 8 bits for the backward pass: SwiGLU and RMSNorm.
// A kept tensor is E4M3 codes and one E8M0 scale per 32 consecutive elements of a row (the layout
// nvfp4_mx_dequantize reads). The scale is the smallest power of two that keeps the block's largest
// magnitude within 448: unlike the MX conversion of mx_kernel.cu nothing saturates, so every normal
// element is off by at most half an E4M3 step (2^-4 of itself).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4_device.cuh"
#include "aux_internal.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr uint32_t kBadOffsets = 0x1u;  // NVFP4_DEVICE_BAD_OFFSETS

// 16 BF16 values of one row: half a block of 32, the other half in the neighbouring lane.
struct Half32 {
  uint4 lo, hi;
};

__device__ __forceinline__ Half32 load_half(const uint4* p) {
  Half32 h;
  h.lo = __ldg(p);
  h.hi = __ldg(p + 1);
  return h;
}
__device__ __forceinline__ void words(const Half32& h, uint32_t (&w)[8]) {
  w[0] = h.lo.x; w[1] = h.lo.y; w[2] = h.lo.z; w[3] = h.lo.w;
  w[4] = h.hi.x; w[5] = h.hi.y; w[6] = h.hi.z; w[7] = h.hi.w;
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
template <int COUNT>
__device__ __forceinline__ uint32_t clean_values(float (&v)[COUNT]) {
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < COUNT; i++) {
    const uint32_t b = (__float_as_uint(v[i]) >> 16) & 0x7FFFu;
    if (b >= 0x7F80u) {
      v[i] = __uint_as_float(0x7FC00000u);
      continue;
    }
    top = max(top, b);
    if (b >= kRoundsToInf) v[i] = copysignf(__uint_as_float(0x7F700000u), v[i]);
  }
  return top;
}

__device__ __forceinline__ uint32_t quad_max(uint32_t m, uint32_t quad) {
  m = max(m, __shfl_xor_sync(quad, m, 1));
  return max(m, __shfl_xor_sync(quad, m, 2));
}

// Codes of the lane's 16 values and the block's scale byte, called by both lanes of a pair
// (lane, lane ^ 1) at once. Scaling by a power of two is exact, so each code is rounded once.
__device__ __forceinline__ uint4 keep_half(const uint32_t (&w)[8], uint32_t& scale) {
  const int lane = threadIdx.x & 31;
  const uint32_t pair = 3u << (lane & 30);
  uint32_t m = abs2(w[0]);
#pragma unroll
  for (int i = 1; i < 8; i++) m = vmax2(m, abs2(w[i]));
  uint32_t top = pair_bits(m);
  top = max(top, __shfl_xor_sync(pair, top, 1));
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
  if (top >= kRoundsToInf) {  // both lanes of the pair
    top = clean_values(v);
    top = max(top, __shfl_xor_sync(pair, top, 1));
  }
  scale = scale_byte(top);
  const float inv = inverse_scale(scale);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; i++)
    c[i] = e4m3x2(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv)) |
           (e4m3x2(__fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv)) << 16);
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// The same for 8 values a lane, the block in the four lanes of a quad: two words of codes.
__device__ __forceinline__ uint2 keep_quarter(const uint32_t (&w)[4], uint32_t& scale) {
  const int lane = threadIdx.x & 31;
  const uint32_t quad = 15u << (lane & 28);
  uint32_t top = pair_bits(vmax2(vmax2(abs2(w[0]), abs2(w[1])), vmax2(abs2(w[2]), abs2(w[3]))));
  top = quad_max(top, quad);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
  if (top >= kRoundsToInf) top = quad_max(clean_values(v), quad);
  scale = scale_byte(top);
  const float inv = inverse_scale(scale);
  uint32_t c[2];
#pragma unroll
  for (int i = 0; i < 2; i++)
    c[i] = e4m3x2(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv)) |
           (e4m3x2(__fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv)) << 16);
  return make_uint2(c[0], c[1]);
}

// The binary32 value of a scale byte (255 is NaN).
__device__ __forceinline__ float e8m0_value(uint32_t s) {
  return s == 0u ? __uint_as_float(0x00400000u)
                 : (s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s << 23));
}

template <int WORDS>
__device__ __forceinline__ void kept_values(const uint32_t (&w)[WORDS], float scale,
                                            float (&v)[4 * WORDS]) {
#pragma unroll
  for (int i = 0; i < 2 * WORDS; i++) {
    const float2 f = e4m3x2_to_float2((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
    v[2 * i] = __fmul_rn(f.x, scale);
    v[2 * i + 1] = __fmul_rn(f.y, scale);
  }
}

// sigmoid(a) from exp(-|a|), which cannot overflow.
__device__ __forceinline__ float sigmoid(float a) {
  const float t = __expf(-fabsf(a));
  const float r = __fdividef(1.0f, __fadd_rn(1.0f, t));
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

__device__ __forceinline__ int64_t live_of(const int32_t* offsets, int32_t E, int64_t M,
                                           uint32_t* status) {
  if (offsets == nullptr) return M;
  const int64_t v = offsets[E - 1];
  if ((v < 0 || v > M) && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, kBadOffsets);
  return v < 0 ? 0 : (v < M ? v : M);
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
    if (blockIdx.x == 0 && offsets && e > 0 && offsets[e] < offsets[e - 1])
      atomicOr(status, kBadOffsets);
  }
  __syncthreads();
  const int64_t nc = F / 16;
  int expert = 0;
  uint32_t m = 0u;
  for (GluWalk it(M, nc, per_cta); it.left > 0; it.next()) {
    const int64_t r = it.row, c = it.col;
    uint4 yo[2], kg = make_uint4(0u, 0u, 0u, 0u), ku = kg;
    uint32_t sg = 0u, su = 0u;
    yo[0] = yo[1] = kg;
    if (r < live) {
      while (expert < E - 1 && r >= ends[expert]) {
        if (m) atomicMax(&top[expert], m);
        m = 0u;
        expert++;
      }
      uint32_t g[8], u[8], o[8];
      words(load_half(h + (r * 2 * nc + c) * 2), g);
      words(load_half(h + (r * 2 * nc + nc + c) * 2), u);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float a0 = bf16_lo(g[i]), a1 = bf16_hi(g[i]);
        o[i] = pack_bf16(__fmul_rn(__fmul_rn(a0, sigmoid(a0)), bf16_lo(u[i])),
                         __fmul_rn(__fmul_rn(a1, sigmoid(a1)), bf16_hi(u[i])));
        m = max(m, pair_bits(abs2(o[i])));
      }
      yo[0] = make_uint4(o[0], o[1], o[2], o[3]);
      yo[1] = make_uint4(o[4], o[5], o[6], o[7]);
      kg = keep_half(g, sg);
      ku = keep_half(u, su);
    }
    y[(r * nc + c) * 2] = yo[0];
    y[(r * nc + c) * 2 + 1] = yo[1];
    codes[r * 2 * nc + c] = kg;
    codes[r * 2 * nc + nc + c] = ku;
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
  const int64_t nc = F / 16;
  for (GluWalk it(M, nc, per_cta); it.left > 0; it.next()) {
    const int64_t r = it.row, c = it.col;
    uint32_t og[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, ou[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (r < live) {
      uint32_t d[8];
      float g[16], u[16];
      words(load_half(grad + (r * nc + c) * 2), d);
      const uint4 kg = __ldg(codes + r * 2 * nc + c), ku = __ldg(codes + r * 2 * nc + nc + c);
      kept_values({kg.x, kg.y, kg.z, kg.w}, e8m0_value(scales[r * nc + c / 2]), g);
      kept_values({ku.x, ku.y, ku.z, ku.w}, e8m0_value(scales[r * nc + nc / 2 + c / 2]), u);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float dg[2], du[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const float dy = j ? bf16_hi(d[i]) : bf16_lo(d[i]);
          const float a = g[2 * i + j], b = u[2 * i + j];
          const float s = sigmoid(a);
          const float slope = __fmul_rn(s, __fmaf_rn(a, __fsub_rn(1.0f, s), 1.0f));
          dg[j] = __fmul_rn(__fmul_rn(dy, b), slope);
          du[j] = __fmul_rn(dy, __fmul_rn(a, s));
        }
        og[i] = pack_bf16(dg[0], dg[1]);
        ou[i] = pack_bf16(du[0], du[1]);
      }
    }
    uint4* pg = grad_h + (r * 2 * nc + c) * 2;
    uint4* pu = grad_h + (r * 2 * nc + nc + c) * 2;
    pg[0] = make_uint4(og[0], og[1], og[2], og[3]);
    pg[1] = make_uint4(og[4], og[5], og[6], og[7]);
    pu[0] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    pu[1] = make_uint4(ou[4], ou[5], ou[6], ou[7]);
  }
}

// ---- RMSNorm -----------------------------------------------------------------------------

// A group of `wpr` warps owns a row, ITEMS x 8 columns a thread (a vector of 16 bytes, neighbouring
// threads neighbouring vectors): the row is read once and stays in registers between its sum and
// its output. A CTA holds as many groups as fit in 16 warps, at least one. With ITEMS = 1 (rows up
// to 8192 columns) the registers also hold the group's next row, which is loaded before the current
// one is summed, so that the SM's loads do not stop at the barrier of the sum.
constexpr int kRmsThreads = 1024;  // of the largest CTA

struct RmsShape {
  int wpr, groups, items;
};
RmsShape rms_shape(int64_t N) {
  RmsShape s;
  s.items = N <= 8192 ? 1 : (N <= 16384 ? 2 : 4);
  const int64_t per_warp = 256 * s.items;
  s.wpr = (int)((N + per_warp - 1) / per_warp);
  s.groups = s.wpr >= 16 ? 1 : 16 / s.wpr;
  return s;
}

// Sum over the group's threads: shuffles, then the warps' sums through shared memory, in an order
// that does not depend on time. `red` has two halves used in turn, so one barrier a row is enough.
__device__ __forceinline__ float group_sum(float s, float (*red)[32], int turn, int group, int wpr) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (wpr == 1) return s;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[turn][threadIdx.x >> 5] = s;
  named_bar_sync(1 + group, wpr * 32);
  s = lane < wpr ? red[turn][group * wpr + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

template <int ITEMS>
__global__ void __launch_bounds__(kRmsThreads, 1) rmsnorm_checkpoint_kernel(
    const uint4* __restrict__ x, const uint4* __restrict__ weight, int64_t M, int32_t N, float eps,
    float bias, int wpr, int groups, uint4* y, uint2* codes, uint8_t* scales, float* rstd,
    uint32_t* amax) {
  __shared__ float red[2][32];
  __shared__ uint32_t top[32];
  pdl_wait();
  pdl_allow_next();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = warp / wpr, at = tid - group * wpr * 32, threads = wpr * 32;
  const int nv = N / 8;
  const int64_t step = (int64_t)gridDim.x * groups;
  constexpr bool kAhead = ITEMS == 1;
  uint32_t m = 0u;
  int turn = 0;
  int64_t r = (int64_t)blockIdx.x * groups + group;
  uint4 next[ITEMS], g[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; j++) {
    next[j] = g[j] = make_uint4(0u, 0u, 0u, 0u);
    const int c = at + j * threads;
    if (c < nv) {
      g[j] = __ldg(weight + c);
      if (r < M) next[j] = __ldg(x + r * nv + c);
    }
  }
  for (; r < M; r += step) {
    uint32_t w[ITEMS][4];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int c = at + j * threads;
      w[j][0] = next[j].x; w[j][1] = next[j].y; w[j][2] = next[j].z; w[j][3] = next[j].w;
      if (kAhead && c < nv && r + step < M) next[j] = __ldg(x + (r + step) * nv + c);
    }
#pragma unroll
    for (int j = 0; j < ITEMS; j++)  // (columns past the row hold zeros)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        s = __fmaf_rn(bf16_lo(w[j][i]), bf16_lo(w[j][i]), s);
        s = __fmaf_rn(bf16_hi(w[j][i]), bf16_hi(w[j][i]), s);
      }
    s = group_sum(s, red, turn, group, wpr);
    turn ^= 1;
    const float rs = __frsqrt_rn(__fadd_rn(__fdiv_rn(s, (float)N), eps));
    if (at == 0) rstd[r] = rs;
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int c = at + j * threads;
      if (c >= nv) break;
      const uint32_t ge[4] = {g[j].x, g[j].y, g[j].z, g[j].w};
      uint32_t o[4], sc;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        o[i] = pack_bf16(__fmul_rn(__fadd_rn(bf16_lo(ge[i]), bias), __fmul_rn(bf16_lo(w[j][i]), rs)),
                         __fmul_rn(__fadd_rn(bf16_hi(ge[i]), bias), __fmul_rn(bf16_hi(w[j][i]), rs)));
        m = vmax2(m, abs2(o[i]));
      }
      y[r * nv + c] = make_uint4(o[0], o[1], o[2], o[3]);
      codes[r * nv + c] = keep_quarter(w[j], sc);
      if ((c & 3) == 0) scales[r * (nv / 4) + c / 4] = (uint8_t)sc;
      if (!kAhead && r + step < M) next[j] = __ldg(x + (r + step) * nv + c);
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
template <int ITEMS, bool RES>
__global__ void __launch_bounds__(kRmsThreads, 1) rmsnorm_checkpoint_backward_kernel(
    const uint4* __restrict__ grad, const uint2* __restrict__ codes,
    const uint8_t* __restrict__ scales, const float* __restrict__ rstd,
    const uint4* __restrict__ weight, int64_t M, int32_t N, float bias, int wpr, int groups,
    const uint4* __restrict__ residual, uint4* grad_x, float* partial) {
  __shared__ float red[2][32];
  __shared__ float4 cols[2048 / 4];  // the groups' joint sums: more than one group has N <= 2048
  pdl_wait();
  pdl_allow_next();
  const int tid = threadIdx.x, warp = tid >> 5;
  const int group = warp / wpr, at = tid - group * wpr * 32, threads = wpr * 32;
  const int nv = N / 8;
  const int64_t step = (int64_t)gridDim.x * groups;
  float dw[ITEMS][8];
#pragma unroll
  for (int j = 0; j < ITEMS; j++)
#pragma unroll
    for (int i = 0; i < 8; i++) dw[j][i] = 0.0f;
  int turn = 0;
  constexpr bool kAhead = ITEMS == 1;
  struct Row {
    uint4 d[ITEMS], res[ITEMS];
    uint2 k[ITEMS];
    uint32_t sc[ITEMS];
    float rs;
  } next;
  auto load = [&](int64_t r) {
    next.rs = rstd[r];
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int c = at + j * threads;
      if (c < nv) {
        next.d[j] = __ldg(grad + r * nv + c);
        next.k[j] = __ldg(codes + r * nv + c);
        next.sc[j] = __ldg(scales + r * (nv / 4) + c / 4);
        if (RES) next.res[j] = __ldg(residual + r * nv + c);
      }
    }
  };
#pragma unroll
  for (int j = 0; j < ITEMS; j++) {
    next.d[j] = next.res[j] = make_uint4(0u, 0u, 0u, 0u);
    next.k[j] = make_uint2(0u, 0u);
    next.sc[j] = 0u;
  }
  int64_t r = (int64_t)blockIdx.x * groups + group;
  if (kAhead && r < M) load(r);
  for (; r < M; r += step) {
    if (!kAhead) load(r);
    const Row row = next;
    if (kAhead && r + step < M) load(r + step);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int c = at + j * threads;
      if (c >= nv) break;
      const uint4 gw = __ldg(weight + c);
      const uint32_t g[4] = {gw.x, gw.y, gw.z, gw.w};
      const uint32_t d[4] = {row.d[j].x, row.d[j].y, row.d[j].z, row.d[j].w};
      float v[8];
      kept_values({row.k[j].x, row.k[j].y}, e8m0_value(row.sc[j]), v);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float dy = (i & 1) ? bf16_hi(d[i >> 1]) : bf16_lo(d[i >> 1]);
        const float w = __fadd_rn((i & 1) ? bf16_hi(g[i >> 1]) : bf16_lo(g[i >> 1]), bias);
        const float t = __fmul_rn(dy, __fmul_rn(v[i], row.rs));
        dw[j][i] = __fadd_rn(dw[j][i], t);
        s = __fmaf_rn(w, t, s);
      }
    }
    s = group_sum(s, red, turn, group, wpr);
    turn ^= 1;
    const float mean = __fdiv_rn(s, (float)N);
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int c = at + j * threads;
      if (c >= nv) break;
      const uint4 gw = __ldg(weight + c);
      const uint32_t g[4] = {gw.x, gw.y, gw.z, gw.w};
      const uint32_t d[4] = {row.d[j].x, row.d[j].y, row.d[j].z, row.d[j].w};
      const uint32_t e[4] = {row.res[j].x, row.res[j].y, row.res[j].z, row.res[j].w};
      uint32_t o[4];
      float v[8];
      kept_values({row.k[j].x, row.k[j].y}, e8m0_value(row.sc[j]), v);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float q[2];
#pragma unroll
        for (int b = 0; b < 2; b++) {
          const float dy = b ? bf16_hi(d[i]) : bf16_lo(d[i]);
          const float w = __fadd_rn(b ? bf16_hi(g[i]) : bf16_lo(g[i]), bias);
          const float xh = __fmul_rn(v[2 * i + b], row.rs);
          q[b] = __fmul_rn(row.rs, __fmaf_rn(-xh, mean, __fmul_rn(w, dy)));
          if (RES) q[b] = __fadd_rn(q[b], b ? bf16_hi(e[i]) : bf16_lo(e[i]));
        }
        o[i] = pack_bf16(q[0], q[1]);
      }
      grad_x[r * nv + c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  float4* out = reinterpret_cast<float4*>(partial + (int64_t)blockIdx.x * N);
  for (int g = 0; g < groups; g++) {
    if (group == g) {
#pragma unroll
      for (int j = 0; j < ITEMS; j++) {
        const int c = at + j * threads;
        if (c >= nv) break;
#pragma unroll
        for (int i = 0; i < 2; i++) {
          float4 v = make_float4(dw[j][4 * i], dw[j][4 * i + 1], dw[j][4 * i + 2], dw[j][4 * i + 3]);
          if (g > 0) {
            const float4 p = cols[c * 2 + i];
            v = make_float4(p.x + v.x, p.y + v.y, p.z + v.z, p.w + v.w);
          }
          if (g == groups - 1) out[c * 2 + i] = v;
          else cols[c * 2 + i] = v;
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

int64_t glu_per_cta(int64_t items, int sm_count, int* grid) {
  const int64_t most = (int64_t)sm_count * 8;
  int64_t per = (items + most - 1) / most;
  per = (per + kGluThreads - 1) / kGluThreads * kGluThreads;
  *grid = (int)((items + per - 1) / per);
  return per;
}

// One wave: the CTAs that the registers of 1024 threads allow on every SM.
int rms_grid(const RmsShape& f, int64_t M, int sm_count) {
  const int64_t ctas = (M + f.groups - 1) / f.groups;
  const int64_t wave = (int64_t)sm_count * (kRmsThreads / (f.wpr * f.groups * 32));
  return (int)(ctas < wave ? ctas : wave);
}

template <int ITEMS>
cudaError_t rms_forward_t(const RmsArgs& a, const RmsShape& f, int sm_count, cudaStream_t s) {
  return launch_pdl(rmsnorm_checkpoint_kernel<ITEMS>, dim3(rms_grid(f, a.M, sm_count)),
                    dim3(f.wpr * f.groups * 32), 0, s, static_cast<const uint4*>(a.x),
                    static_cast<const uint4*>(a.weight), a.M, (int32_t)a.N, a.eps, a.bias, f.wpr,
                    f.groups, static_cast<uint4*>(a.y), static_cast<uint2*>(a.codes), a.scales,
                    a.rstd, reinterpret_cast<uint32_t*>(a.amax));
}

template <int ITEMS>
cudaError_t rms_backward_t(const RmsArgs& a, const RmsShape& f, int sm_count, cudaStream_t s) {
  int grid = rms_grid(f, a.M, sm_count);
  if (grid > kRmsMaxPartials) grid = kRmsMaxPartials;
  const cudaError_t e = launch_pdl(
      a.residual ? rmsnorm_checkpoint_backward_kernel<ITEMS, true>
                 : rmsnorm_checkpoint_backward_kernel<ITEMS, false>,
      dim3(grid), dim3(f.wpr * f.groups * 32), 0, s, static_cast<const uint4*>(a.grad),
      static_cast<const uint2*>(a.codes), a.scales, a.rstd, static_cast<const uint4*>(a.weight),
      a.M, (int32_t)a.N, a.bias, f.wpr, f.groups, static_cast<const uint4*>(a.residual),
      static_cast<uint4*>(a.grad_x), a.partial);
  if (e != cudaSuccess) return e;
  return launch_pdl(column_sum_kernel, dim3((unsigned)(a.N / 32)), dim3(32 * kSumWarps), 0, s,
                    a.partial, grid, a.N, a.grad_weight);
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

cudaError_t launch_rmsnorm_checkpoint(const RmsArgs& a, int sm_count, cudaStream_t s) {
  const RmsShape f = rms_shape(a.N);
  if (f.items == 1) return rms_forward_t<1>(a, f, sm_count, s);
  if (f.items == 2) return rms_forward_t<2>(a, f, sm_count, s);
  return rms_forward_t<4>(a, f, sm_count, s);
}

cudaError_t launch_rmsnorm_checkpoint_backward(const RmsArgs& a, int sm_count, cudaStream_t s) {
  const RmsShape f = rms_shape(a.N);
  if (f.items == 1) return rms_backward_t<1>(a, f, sm_count, s);
  if (f.items == 2) return rms_backward_t<2>(a, f, sm_count, s);
  return rms_backward_t<4>(a, f, sm_count, s);
}

}  // namespace nvfp4
