// The owner's walk over a ring of tiles (csrc/tile_ring.h) on simulated barriers: phases complete
// when the copy that belongs to them lands, and a wait moves time on by at most its limit.
#include <cstdint>
#include <vector>

#include "tile_ring.h"

namespace {

constexpr int64_t kLimit = 100;

struct Copy {
  int stage, tile;
  int64_t lands;  // < 0: never
};

template <int STAGES>
struct Sim {
  int64_t now = 0;
  std::vector<Copy> flying;
  int done[STAGES] = {};  // completed phases of each barrier
  int held[STAGES];       // the tile that a buffer holds
  int timeouts = 0, idle_timeouts = 0;

  void land() {
    for (size_t i = 0; i < flying.size();) {
      const Copy c = flying[i];
      if (c.lands >= 0 && c.lands <= now) {
        done[c.stage]++;
        held[c.stage] = c.tile;
        flying.erase(flying.begin() + i);
      } else {
        i++;
      }
    }
  }
  bool wait(int stage, uint32_t parity) {
    for (int64_t t = 0; t <= kLimit; t++, now++) {
      land();
      if ((uint32_t)(done[stage] & 1) != parity) return true;  // as mbarrier.try_wait.parity
    }
    timeouts++;
    bool any = false;
    for (const Copy& c : flying) any = any || c.stage == stage;
    if (!any) idle_timeouts++;
    return false;
  }
};

// out: {tile at which the owner gave up (-1), copies in flight when it leaves, waits that ran out,
// those of them on a barrier without a copy in flight, tiles that were read with other contents}
template <int STAGES>
void run(int tiles, const int64_t* delay, int64_t* out) {
  Sim<STAGES> sim;
  nvfp4::TileRing<STAGES> ring;
  for (int i = 0; i < STAGES; i++) sim.held[i] = -1;
  auto fetch = [&](int stage, int tile) {
    if (tile >= tiles) return;
    sim.flying.push_back({stage, tile, delay[tile] < 0 ? -1 : sim.now + delay[tile]});
  };
  int64_t gave_up = -1, wrong = 0;
  for (int i = 0; i < ring.kAhead; i++) fetch(i, i);
  for (int t = 0; t < tiles; t++) {
    const bool was = ring.dead;
    ring.wait(true, [&](int s, uint32_t p) { return sim.wait(s, p); },
              [&](int i) { return t + i < tiles; });
    if (ring.dead && !was) gave_up = t;
    if (!ring.dead && sim.held[ring.stage] != t) wrong++;
    if (STAGES > 1 && !ring.dead)
      fetch(ring.stage == 0 ? STAGES - 1 : ring.stage - 1, t + STAGES - 1);
    ring.next();
    if (STAGES == 1 && !ring.dead) fetch(0, t + 1);
  }
  sim.land();
  out[0] = gave_up;
  out[1] = (int64_t)sim.flying.size();
  out[2] = sim.timeouts;
  out[3] = sim.idle_timeouts;
  out[4] = wrong;
}

}  // namespace

// delay[tile]: how long after its fetch a tile's copy lands (limit of a wait: 100), -1 never.
extern "C" int tile_ring_sim(int stages, int tiles, const int64_t* delay, int64_t* out) {
  switch (stages) {
    case 1: run<1>(tiles, delay, out); return 0;
    case 2: run<2>(tiles, delay, out); return 0;
    case 3: run<3>(tiles, delay, out); return 0;
    case 4: run<4>(tiles, delay, out); return 0;
  }
  return 1;
}
