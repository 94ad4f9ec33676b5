// cache.cuh -- device helpers of the paged-cache kernels.
#pragma once
#include <cuda_runtime.h>

#include "serving.h"

namespace ra {

// First error of a cache call into the workspace's error word.
__device__ __forceinline__ void record_cache_fault(uint32_t* err, int kernel_id, int what, int b) {
  if (atomicCAS(err, 0u, (uint32_t)RA_ERR_CACHE) == 0u) {
    err[1] = (uint32_t)kernel_id;
    err[2] = (uint32_t)what;
    err[3] = (uint32_t)b;
  }
}

// Page of sequence b that holds the 16-token block `blk`, or -1 (recorded) if its table entry
// lies outside the cache.
__device__ __forceinline__ int page_of(const CacheDims& c, const int* __restrict__ table, int b,
                                       int blk, uint32_t* err, int kernel_id) {
  const int page = table[(long long)b * c.max_pages + blk / c.page_blocks];
  if (page_ok(c, page)) return page;
  record_cache_fault(err, kernel_id, RA_CACHE_BAD_PAGE, b);
  return -1;
}

}  // namespace ra
