// Test-only: the tile ring of csrc/tile_ring.h on the GPU, one CTA, with the copy of one tile left
// out, so that the waits for it run out after a short limit and the kernel reports it and ends.
#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4_device.cuh"
#include "tile_ring.h"

namespace {

using namespace nvfp4;

constexpr int kThreads = 64;
constexpr int kWords = kThreads;  // 32-bit words of a tile, one a thread
constexpr uint64_t kLimitNs = 20000000ull;

// seen[tile][thread]: the word read, or ~0 for a thread that has given up. info: [0] tile at which
// thread 0 gave up (-1), [1] copies that it issued, [2] those whose phase is complete at the end,
// [3] threads that gave up.
template <int STAGES>
__global__ void ring_kernel(const uint32_t* src, int tiles, int dropped, uint32_t* seen,
                            int* info) {
  __shared__ __align__(128) uint32_t ring[STAGES][kWords];
  __shared__ __align__(8) uint64_t full[STAGES];
  const int tid = threadIdx.x;
  if (tid == 0) {
    for (int i = 0; i < STAGES; i++) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  int issued[STAGES] = {}, last_dropped = -1;
  auto fetch = [&](int stage, int tile) {  // thread 0
    if (tile >= tiles) return;
    mbar_expect_tx(&full[stage], kWords * 4);
    issued[stage]++;
    if (tile == dropped) last_dropped = stage;
    else bulk_load(ring[stage], src + tile * kWords, kWords * 4, &full[stage]);
  };
  TileRing<STAGES> at;
  if (tid == 0) {
    info[0] = -1;
    for (int i = 0; i < at.kAhead; i++) fetch(i, i);
  }
  for (int t = 0; t < tiles; t++) {
    const bool was = at.dead;
    at.wait(tid == 0,
            [&](int stage, uint32_t parity) {
              return mbar_wait_bounded(&full[stage], parity, kLimitNs);
            },
            [&](int i) { return t + i < tiles; });
    if (tid == 0 && at.dead && !was) info[0] = t;
    seen[t * kThreads + tid] = at.dead ? ~0u : ring[at.stage][tid];
    __syncthreads();
    if (STAGES > 1 && tid == 0 && !at.dead)
      fetch(at.stage == 0 ? STAGES - 1 : at.stage - 1, t + STAGES - 1);
    at.next();
    if (STAGES == 1 && tid == 0 && !at.dead) fetch(0, t + 1);
  }
  if (at.dead) atomicAdd(&info[3], 1);
  if (tid == 0)
    for (int i = 0; i < STAGES; i++) {
      info[1] += issued[i] - (i == last_dropped);
      if (issued[i] > 0 && i != last_dropped)
        info[2] += mbar_try_wait(&full[i], (issued[i] - 1) & 1) ? issued[i] : 0;
      else if (i == last_dropped)
        info[2] += issued[i] - 1;  // its earlier copies were waited for
    }
}

}  // namespace

// Device pointers: src [tiles][64] words, seen [tiles][64], info [4] zeroed. dropped -1: none.
extern "C" int probe_tile_ring(int stages, int tiles, int dropped, const void* src, void* seen,
                               void* info, void* stream) {
  auto* s = static_cast<const uint32_t*>(src);
  auto* o = static_cast<uint32_t*>(seen);
  auto* n = static_cast<int*>(info);
  auto st = static_cast<cudaStream_t>(stream);
  switch (stages) {
    case 1: ring_kernel<1><<<1, kThreads, 0, st>>>(s, tiles, dropped, o, n); break;
    case 2: ring_kernel<2><<<1, kThreads, 0, st>>>(s, tiles, dropped, o, n); break;
    case 3: ring_kernel<3><<<1, kThreads, 0, st>>>(s, tiles, dropped, o, n); break;
    case 4: ring_kernel<4><<<1, kThreads, 0, st>>>(s, tiles, dropped, o, n); break;
    default: return -1;
  }
  return (int)cudaGetLastError();
}
