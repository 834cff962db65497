// Drives the ring of csrc/kvb_ring.h against a model of its barriers: a barrier counts completed phases, and a
// wait on parity p passes when the phase being filled has the other parity.  A warp leaves before each possible
// step; the drain has to wait for every copy in flight and for nothing else.  Prints the cases looked at.
#include <cstdio>
#include <vector>

#include "kvb_ring.h"

using namespace w4::kvb;

template <int S>
static int cases() {
  int n = 0;
  for (int steps = 0; steps <= 5 * S + 1; ++steps)
    for (int left = 0; left <= steps; ++left, ++n) {
      std::vector<int> done(S, 0), flying(S, 0);  // phases completed; copies in flight
      auto passes = [&](int stage, uint32_t parity) { return ((uint32_t)done[stage] & 1u) != parity; };
      auto issue = [&](int k) {
        if (k >= steps) return true;
        const int stage = ring_stage<S>(k);
        if (flying[stage]) return false;  // over a copy in flight
        flying[stage] = 1;
        return true;
      };
      auto land = [&](int stage) {
        flying[stage] = 0;
        ++done[stage];
      };
      for (int k = 0; k < S; ++k)
        if (!issue(k)) return -1;
      for (int k = 0; k < left; ++k) {  // the steps that the warp reads
        const int stage = ring_stage<S>(k);
        if (passes(stage, ring_parity<S>(k))) return -2;  // before its copies have landed
        land(stage);
        if (!passes(stage, ring_parity<S>(k))) return -3;
        if (!issue(k + S)) return -4;
      }
      int waits = 0, flew = 0;
      for (int stage = 0; stage < S; ++stage) flew += flying[stage];
      bool bad = false;
      ring_drain<S>(left, steps, [&](int stage, uint32_t parity) {
        ++waits;
        bad |= !flying[stage] || passes(stage, parity);  // nothing to wait for, or not waited for
        land(stage);
        bad |= !passes(stage, parity);  // a wait without an end
      });
      if (bad || waits != flew) return -5;
    }
  return n;
}

int main() {
  const int a = cases<2>(), b = cases<3>(), c = cases<4>();
  std::printf("%d %d %d\n", a, b, c);
  return a < 0 || b < 0 || c < 0;
}
