// A warp's ring of S stages, each with one barrier: step k fills and reads stage
// k % S.  Plain C++, so that the arithmetic can be tested without a GPU.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define KVB_RING_FN __host__ __device__ __forceinline__
#else
#define KVB_RING_FN inline
#endif

namespace w4 {
namespace kvb {

// Stage of step k, and the parity of the barrier's phase that its copies complete.
template <int S>
KVB_RING_FN int ring_stage(int k) {
  return k % S;
}
template <int S>
KVB_RING_FN uint32_t ring_parity(int k) {
  return (uint32_t)(k / S) & 1u;
}

// Every copy in flight, for a warp that left its loop of `steps` steps before reading step `left`
// (`steps`: it read them all): those of steps left .. left + S - 1, each on its own phase.  wait(stage, parity).
template <int S, typename Wait>
KVB_RING_FN void ring_drain(int left, int steps, Wait&& wait) {
  for (int k = left; k < steps && k < left + S; ++k) wait(ring_stage<S>(k), ring_parity<S>(k));
}

}  // namespace kvb
}  // namespace w4
