// toplist.cuh -- a row's largest elements as a warp's sorted list of 32 keys, lane j holding the
// j-th (order key of the logit, then the complement of the index: a larger key is a larger
// logit or, on a tie, a lower index).
#pragma once

#include "common.cuh"

namespace svk {

// 64-bit keys held one per lane, sorted descending by a bitonic network (blocks of
// size s alternate direction so that each pair forms a bitonic sequence; size 32 is
// descending).
__device__ __forceinline__ uint64_t warp_sort_desc(uint64_t x, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const uint64_t y = __shfl_xor_sync(kFull, x, stride);
      const bool desc = (lane & size) == 0, low = (lane & stride) == 0;
      x = (low == desc) ? (x > y ? x : y) : (x < y ? x : y);
    }
  }
  return x;
}

// The list with one key more.  Only its first k_out places matter.
__device__ __forceinline__ uint64_t list_insert(uint64_t L, uint64_t x, int k_out, int lane) {
  const int pos = __popc(__ballot_sync(kFull, L > x));
  if (pos < k_out) {
    const uint64_t up = __shfl_up_sync(kFull, L, 1);
    if (lane > pos) L = up;
    if (lane == pos) L = x;
  }
  return L;
}

// The list merged with another list: reversed against it, the lane-wise larger of the two are
// the 32 largest of both, as a bitonic sequence, which one more network sorts.
__device__ __forceinline__ uint64_t list_merge(uint64_t L, uint64_t x, int lane) {
  const uint64_t y = __shfl_sync(kFull, x, 31 - lane);
  L = L > y ? L : y;
#pragma unroll
  for (int stride = 16; stride > 0; stride >>= 1) {
    const uint64_t o = __shfl_xor_sync(kFull, L, stride);
    L = ((lane & stride) == 0) == (L > o) ? L : o;
  }
  return L;
}

}  // namespace svk
