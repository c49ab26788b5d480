// paged.cuh -- addressing of a paged key / value cache, shared by the append, attention
// and commit kernels.
//
// A sequence's position t lives in slot t % page_size of page table[t / page_size].  A
// page number outside [0, n_pages) holds nothing: keys there are masked, tokens are not
// written and rows are not moved, so a stale or padded table entry never leads to an
// access outside the cache.
#pragma once

#include "common.cuh"

namespace svk {

// x / d by a multiplication: the high half of x * ceil(2^64 / d) is exact for x below 2^32.
struct FastDiv {
  uint64_t magic;
  int d;
  __host__ static FastDiv make(int d) {
    return FastDiv{d > 1 ? ~0ull / (uint64_t)d + 1u : 0u, d};
  }
  __device__ __forceinline__ int div(int x) const {
    return d == 1 ? x : (int)__umul64hi((uint64_t)(uint32_t)x, magic);
  }
};

// t / page_size and t % page_size; `shift` >= 0 for a power of two.
struct PageDiv {
  int32_t size, shift;
  __host__ static PageDiv make(int32_t page_size) {
    PageDiv d{page_size, -1};
    if ((page_size & (page_size - 1)) == 0)
      for (d.shift = 0; (1 << d.shift) < page_size;) ++d.shift;
    return d;
  }
  __device__ __forceinline__ int div(int t) const { return shift >= 0 ? t >> shift : t / size; }
};

// Offset of position t's row (in the unit of the strides, 64-bit: a long cache passes 32
// bits), or -1 where the table or the page number has no such position.
__device__ __forceinline__ int64_t paged_offset(const int32_t* table_row, int max_pages,
                                                int n_pages, PageDiv pd, int64_t page_stride,
                                                int64_t pos_stride, int t) {
  if (t < 0) return -1;
  const int at = pd.div(t);
  if (at >= max_pages) return -1;
  const int page = table_row[at];
  if ((unsigned)page >= (unsigned)n_pages) return -1;
  return (int64_t)page * page_stride + (int64_t)(t - at * pd.size) * pos_stride;
}

// Host checks of a paged cache's sizes (append.cu): SPEC_OK or an error code.
int check_paged_layout(const spec_paged_layout& l, int32_t max_pages);

}  // namespace svk
