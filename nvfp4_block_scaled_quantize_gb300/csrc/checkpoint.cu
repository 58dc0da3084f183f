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

// Codes of the lane's 16 values and the block's scale byte. With a = 2^(E-127) (1 + m/128) the
// block's largest BF16 magnitude, a <= 448 * 2^e = 1.75 * 2^(8+e) first holds at e = E - 127 - 8
// when m <= 96 and one above it otherwise, so the biased scale is ((bits + 31) >> 7) - 8, at least
// 0. Scaling by a power of two is exact, so each code is rounded once. Infinities and NaN do not
// count for the maximum and become E4M3 NaN (E4M3 has no infinity), so they reach the gradient.
// Finite magnitudes from 1.9375 * 2^127 up would round to 2^128, outside binary32: they are kept
// as 1.875 * 2^127, so that what is finite stays finite. Called by both lanes of a pair (lane, lane ^ 1) at once.
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
    top = 0u;
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const uint32_t b = (__float_as_uint(v[i]) >> 16) & 0x7FFFu;
      if (b >= 0x7F80u) {
        v[i] = __uint_as_float(0x7FC00000u);
        continue;
      }
      top = max(top, b);
      if (b >= kRoundsToInf) v[i] = copysignf(__uint_as_float(0x7F700000u), v[i]);
    }
    top = max(top, __shfl_xor_sync(pair, top, 1));
  }
  const uint32_t biased = (top + 31u) >> 7;
  scale = biased > 8u ? biased - 8u : 0u;
  const float inv = __uint_as_float((254u - scale) << 23);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; i++)
    c[i] = e4m3x2(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv)) |
           (e4m3x2(__fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv)) << 16);
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// The binary32 value of a scale byte (255 is NaN).
__device__ __forceinline__ float e8m0_value(uint32_t s) {
  return s == 0u ? __uint_as_float(0x00400000u)
                 : (s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s << 23));
}

__device__ __forceinline__ void kept_values(const uint4& c, float scale, float (&v)[16]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 8; i++) {
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
      kept_values(__ldg(codes + r * 2 * nc + c), e8m0_value(scales[r * nc + c / 2]), g);
      kept_values(__ldg(codes + r * 2 * nc + nc + c),
                  e8m0_value(scales[r * nc + nc / 2 + c / 2]), u);
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

// A group of WPR warps owns a row, ITEMS x 16 columns a thread: the row is read once and stays in
// registers between its sum and its output. A CTA of 16 warps holds 16 / WPR groups.
constexpr int kRmsWarps = 16;
constexpr int kRmsThreads = 32 * kRmsWarps;

// Sum over the group's threads: shuffles, then the warps' sums in order. `red` has two halves used
// in turn, so one barrier a row is enough.
template <int WPR>
__device__ __forceinline__ float group_sum(float s, float (*red)[kRmsWarps], int turn) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (WPR == 1) return s;
  const int warp = threadIdx.x >> 5, group = warp / WPR;
  if ((threadIdx.x & 31) == 0) red[turn][warp] = s;
  named_bar_sync(1 + group, WPR * 32);
  s = red[turn][group * WPR];
#pragma unroll
  for (int i = 1; i < WPR; i++) s += red[turn][group * WPR + i];
  return s;
}

template <int WPR, int ITEMS>
__global__ void __launch_bounds__(kRmsThreads) rmsnorm_checkpoint_kernel(
    const uint4* __restrict__ x, const uint4* __restrict__ weight, int64_t M, int64_t N, float eps,
    float bias, uint4* y, uint4* codes, uint8_t* scales, float* rstd, uint32_t* amax) {
  __shared__ float red[2][kRmsWarps];
  __shared__ uint32_t top[kRmsWarps];
  pdl_wait();
  pdl_allow_next();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = warp / WPR, at = tid - group * WPR * 32;
  const int64_t nc = N / 16;
  constexpr int kGroups = kRmsWarps / WPR;
  uint32_t m = 0u;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * kGroups + group; r < M; r += (int64_t)gridDim.x * kGroups) {
    uint32_t w[ITEMS][8];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int64_t c = at + j * WPR * 32;
      if (c < nc) words(load_half(x + (r * nc + c) * 2), w[j]);
    }
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      if (at + j * WPR * 32 >= nc) break;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        s = __fmaf_rn(bf16_lo(w[j][i]), bf16_lo(w[j][i]), s);
        s = __fmaf_rn(bf16_hi(w[j][i]), bf16_hi(w[j][i]), s);
      }
    }
    s = group_sum<WPR>(s, red, turn);
    turn ^= 1;
    const float rs = __frsqrt_rn(__fadd_rn(__fdiv_rn(s, (float)N), eps));
    if (at == 0) rstd[r] = rs;
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int64_t c = at + j * WPR * 32;
      if (c >= nc) break;
      uint32_t g[8], o[8], sc;
      words(load_half(weight + c * 2), g);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        o[i] = pack_bf16(__fmul_rn(__fadd_rn(bf16_lo(g[i]), bias), __fmul_rn(bf16_lo(w[j][i]), rs)),
                         __fmul_rn(__fadd_rn(bf16_hi(g[i]), bias), __fmul_rn(bf16_hi(w[j][i]), rs)));
        m = max(m, pair_bits(abs2(o[i])));
      }
      y[(r * nc + c) * 2] = make_uint4(o[0], o[1], o[2], o[3]);
      y[(r * nc + c) * 2 + 1] = make_uint4(o[4], o[5], o[6], o[7]);
      codes[r * nc + c] = keep_half(w[j], sc);
      if ((c & 1) == 0) scales[r * (nc / 2) + c / 2] = (uint8_t)sc;
    }
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (lane == 0) top[warp] = m;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kRmsWarps; i++) m = max(m, top[i]);
    atomicMax(amax, m << 16);
  }
}

// With xh = x * rstd and g = (w + bias) dy: dx = rstd (g - xh mean(g xh)) [+ residual], and
// dw = sum over rows of dy xh. A thread keeps its columns' share of dw over all of its rows; the
// groups of a CTA are added in shared memory in order and each CTA writes one row of `partial`, so
// that the sum's order depends on the grid alone.
template <int WPR, int ITEMS, bool RES>
__global__ void __launch_bounds__(kRmsThreads, 1) rmsnorm_checkpoint_backward_kernel(
    const uint4* __restrict__ grad, const uint4* __restrict__ codes,
    const uint8_t* __restrict__ scales, const float* __restrict__ rstd,
    const uint4* __restrict__ weight, int64_t M, int64_t N, float bias,
    const uint4* __restrict__ residual, uint4* grad_x, float* partial) {
  constexpr int kGroups = kRmsWarps / WPR;
  __shared__ float red[2][kRmsWarps];
  __shared__ float4 cols[kGroups > 1 ? WPR * 32 * ITEMS * 4 : 1];
  pdl_wait();
  pdl_allow_next();
  const int tid = threadIdx.x, warp = tid >> 5;
  const int group = warp / WPR, at = tid - group * WPR * 32;
  const int64_t nc = N / 16;
  float dw[ITEMS][16];
#pragma unroll
  for (int j = 0; j < ITEMS; j++)
#pragma unroll
    for (int i = 0; i < 16; i++) dw[j][i] = 0.0f;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * kGroups + group; r < M; r += (int64_t)gridDim.x * kGroups) {
    uint32_t d[ITEMS][8], res[ITEMS][8];
    uint4 k[ITEMS];
    float sc[ITEMS];
    const float rs = rstd[r];
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int64_t c = at + j * WPR * 32;
      if (c < nc) {
        words(load_half(grad + (r * nc + c) * 2), d[j]);
        k[j] = __ldg(codes + r * nc + c);
        sc[j] = e8m0_value(scales[r * (nc / 2) + c / 2]);
        if (RES) words(load_half(residual + (r * nc + c) * 2), res[j]);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int64_t c = at + j * WPR * 32;
      if (c >= nc) break;
      uint32_t g[8];
      float v[16];
      words(load_half(weight + c * 2), g);
      kept_values(k[j], sc[j], v);
#pragma unroll
      for (int i = 0; i < 16; i++) {
        const float dy = (i & 1) ? bf16_hi(d[j][i >> 1]) : bf16_lo(d[j][i >> 1]);
        const float w = __fadd_rn((i & 1) ? bf16_hi(g[i >> 1]) : bf16_lo(g[i >> 1]), bias);
        const float t = __fmul_rn(dy, __fmul_rn(v[i], rs));
        dw[j][i] = __fadd_rn(dw[j][i], t);
        s = __fmaf_rn(w, t, s);
      }
    }
    s = group_sum<WPR>(s, red, turn);
    turn ^= 1;
    const float mean = __fdiv_rn(s, (float)N);
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
      const int64_t c = at + j * WPR * 32;
      if (c >= nc) break;
      uint32_t g[8], o[8];
      float v[16];
      words(load_half(weight + c * 2), g);
      kept_values(k[j], sc[j], v);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float q[2];
#pragma unroll
        for (int b = 0; b < 2; b++) {
          const float dy = b ? bf16_hi(d[j][i]) : bf16_lo(d[j][i]);
          const float w = __fadd_rn(b ? bf16_hi(g[i]) : bf16_lo(g[i]), bias);
          const float xh = __fmul_rn(v[2 * i + b], rs);
          q[b] = __fmul_rn(rs, __fmaf_rn(-xh, mean, __fmul_rn(w, dy)));
          if (RES) q[b] = __fadd_rn(q[b], b ? bf16_hi(res[j][i]) : bf16_lo(res[j][i]));
        }
        o[i] = pack_bf16(q[0], q[1]);
      }
      grad_x[(r * nc + c) * 2] = make_uint4(o[0], o[1], o[2], o[3]);
      grad_x[(r * nc + c) * 2 + 1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
  float4* out = reinterpret_cast<float4*>(partial + (int64_t)blockIdx.x * N);
#pragma unroll 1
  for (int g = 0; g < kGroups; g++) {
    if (group == g) {
#pragma unroll
      for (int j = 0; j < ITEMS; j++) {
        const int64_t c = at + j * WPR * 32;
        if (c >= nc) break;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float4 v = make_float4(dw[j][4 * i], dw[j][4 * i + 1], dw[j][4 * i + 2], dw[j][4 * i + 3]);
          if (kGroups > 1) {
            if (g > 0) {
              const float4 p = cols[c * 4 + i];
              v = make_float4(p.x + v.x, p.y + v.y, p.z + v.z, p.w + v.w);
            }
            cols[c * 4 + i] = v;
          }
          if (g == kGroups - 1) out[c * 4 + i] = v;
        }
      }
    }
    if (kGroups > 1) __syncthreads();
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

template <int WPR, int ITEMS>
cudaError_t rms_forward_t(const RmsArgs& a, int sm_count, cudaStream_t s) {
  const int64_t groups = kRmsWarps / WPR;
  const int64_t ctas = (a.M + groups - 1) / groups;
  const int grid = (int)(ctas < sm_count ? ctas : sm_count);
  return launch_pdl(rmsnorm_checkpoint_kernel<WPR, ITEMS>, dim3(grid), dim3(kRmsThreads), 0, s,
                    static_cast<const uint4*>(a.x), static_cast<const uint4*>(a.weight), a.M, a.N,
                    a.eps, a.bias, static_cast<uint4*>(a.y), static_cast<uint4*>(a.codes),
                    a.scales, a.rstd, reinterpret_cast<uint32_t*>(a.amax));
}

template <int WPR, int ITEMS>
cudaError_t rms_backward_t(const RmsArgs& a, int sm_count, cudaStream_t s) {
  const int64_t groups = kRmsWarps / WPR;
  const int64_t ctas = (a.M + groups - 1) / groups;
  int grid = (int)(ctas < sm_count ? ctas : sm_count);
  if (grid > kRmsMaxPartials) grid = kRmsMaxPartials;
  const cudaError_t e = launch_pdl(
      a.residual ? rmsnorm_checkpoint_backward_kernel<WPR, ITEMS, true>
                 : rmsnorm_checkpoint_backward_kernel<WPR, ITEMS, false>,
      dim3(grid), dim3(kRmsThreads), 0, s, static_cast<const uint4*>(a.grad),
      static_cast<const uint4*>(a.codes), a.scales, a.rstd, static_cast<const uint4*>(a.weight),
      a.M, a.N, a.bias, static_cast<const uint4*>(a.residual), static_cast<uint4*>(a.grad_x),
      a.partial);
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
  if (a.N <= 512) return rms_forward_t<1, 1>(a, sm_count, s);
  if (a.N <= 1024) return rms_forward_t<1, 2>(a, sm_count, s);
  if (a.N <= 2048) return rms_forward_t<2, 2>(a, sm_count, s);
  if (a.N <= 4096) return rms_forward_t<4, 2>(a, sm_count, s);
  if (a.N <= 8192) return rms_forward_t<8, 2>(a, sm_count, s);
  if (a.N <= 16384) return rms_forward_t<16, 2>(a, sm_count, s);
  return rms_forward_t<16, 4>(a, sm_count, s);
}

cudaError_t launch_rmsnorm_checkpoint_backward(const RmsArgs& a, int sm_count, cudaStream_t s) {
  if (a.N <= 512) return rms_backward_t<1, 1>(a, sm_count, s);
  if (a.N <= 1024) return rms_backward_t<1, 2>(a, sm_count, s);
  if (a.N <= 2048) return rms_backward_t<2, 2>(a, sm_count, s);
  if (a.N <= 4096) return rms_backward_t<4, 2>(a, sm_count, s);
  if (a.N <= 8192) return rms_backward_t<8, 2>(a, sm_count, s);
  if (a.N <= 16384) return rms_backward_t<16, 2>(a, sm_count, s);
  return rms_backward_t<16, 4>(a, sm_count, s);
}

}  // namespace nvfp4
