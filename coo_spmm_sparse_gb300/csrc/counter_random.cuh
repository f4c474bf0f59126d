// Counter-based random numbers: SplitMix64 (Steele, Lea, Flood, OOPSLA 2014)
// as a function of a seed and a draw's number, so that a mask can be made
// again wherever it is needed and is never stored.
#pragma once

#include <cstdint>

namespace snack {

constexpr uint64_t kSplitMixStep = 0x9E3779B97F4A7C15ull;

__device__ __forceinline__ uint64_t splitmix_finish(uint64_t z) {
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

// Draw number t of a seed.
__device__ __forceinline__ uint64_t splitmix(uint64_t seed, uint64_t t) {
  return splitmix_finish(seed + (t + 1ull) * kSplitMixStep);
}

// Sixteen bits decide about an element, so that a draw serves four: at 32 bits
// an element the generator's integer work (about 24 instructions a draw) would
// bind a 16-bit dropout before the memory does.
__device__ __forceinline__ uint32_t draw_lane(uint64_t z, uint32_t lane) {
  return (uint32_t)(z >> (16 * lane)) & 0xffffu;
}

}  // namespace snack
