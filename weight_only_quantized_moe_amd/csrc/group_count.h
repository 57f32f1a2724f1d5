// Counting the ids of groups, a wave of 64 ids at a time.
#pragma once
#include "device_common.h"

namespace hmoe {

// group of an id: ids outside [0, G) are dropped (-1) or the group behind the last
__device__ __forceinline__ int sort_key(int id, int G, int groups) {
  return (unsigned)id < (unsigned)G ? id : (groups > G ? G : -1);
}

// lanes of the wave with the same group as this one (0: none), from ballots over the bits
__device__ __forceinline__ uint64_t same_group(int e, int bits) {
  uint64_t m = __ballot(e >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool bit = (e >> b) & 1;
    const uint64_t bb = __ballot(bit);
    m &= bit ? bb : ~bb;
  }
  return e >= 0 ? m : 0;
}

__device__ __forceinline__ int group_bits(int groups) { return groups > 1 ? 32 - __clz(groups - 1) : 0; }

// adds the wave's ids to a counter per group: one LDS operation a group, not one a lane
// (few groups would make 64 lanes wait for one address)
__device__ __forceinline__ void count_groups(int e, int bits, int32_t* s_cnt) {
  const uint64_t m = same_group(e, bits);
  if (m && __ffsll((unsigned long long)m) - 1 == (int)(threadIdx.x & (kWave - 1)))
    atomicAdd(&s_cnt[e], __popcll(m));
}

}  // namespace hmoe
