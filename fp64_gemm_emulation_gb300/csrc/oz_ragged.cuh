// oz_ragged.cuh -- row offsets of groups, read on the device.
#pragma once

#include <cstdint>

namespace oz {

// The offsets of `groups` groups of rows into off[0 .. groups] (shared memory), clamped to [0, rows] and to
// their predecessors, so that no access leaves the matrices whatever they hold; given == nullptr: one
// group of all rows.  Called by one whole warp.  Returns whether one had to be clamped.
__device__ __forceinline__ bool clamp_offsets(const int32_t* given, int groups, int rows, int* off) {
  const int lane = threadIdx.x & 31;
  if (!given) {
    if (lane < 2) off[lane] = lane * rows;
    return false;
  }
  int before = 0;
  bool bad = false;
  for (int b = 0; b <= groups; b += 32) {
    const int i = b + lane;
    const int g = i <= groups ? given[i] : 0;
    int v = max(0, min(g, rows));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v = max(v, o);
    }
    v = max(v, before);
    bad |= i <= groups && v != g;
    before = __shfl_sync(0xFFFFFFFFu, v, 31);
    if (i <= groups) off[i] = v;
  }
  return __any_sync(0xFFFFFFFFu, bad);
}

// The last group whose first[group] <= i, for i >= first[0]: first holds groups + 1 ascending values.
__device__ __forceinline__ int group_of(const int* first, int groups, int i) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// Column blocks (128 rows of one column) start anew with each group: group e's first block has this number
// and its rows lie from 128 times that on, rounded up to whole blocks.  The blocks of two groups never meet:
// ceil(l / 128) <= floor((o + l) / 128) - floor(o / 128) + 1 for a group of l rows from row o on.
constexpr int kScaleBlock = 128;
__host__ __device__ inline int first_column_block(int offset, int group) { return offset / kScaleBlock + group; }
__host__ __device__ inline int column_blocks(int rows, int groups, bool ragged) {
  return ragged ? rows / kScaleBlock + groups : rows / kScaleBlock + (rows % kScaleBlock != 0);
}

}  // namespace oz
