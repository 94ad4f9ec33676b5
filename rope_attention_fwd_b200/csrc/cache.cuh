// cache.cuh -- device helpers of the paged-cache kernels.
#pragma once
#include <cuda_fp16.h>
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

// lo + step * code of a word's eight codes, rounded once.  Four bits alone are an fp16 subnormal,
// c 2^-24 or (bits 4-7) c 2^-20, two of them in a masked word; the powers of two go into the step
// (all exact).
__device__ __forceinline__ void codes_to_values(uint32_t w, float step, float lo, float (&x)[8]) {
  const float even = step * 16777216.f, odd = step * 1048576.f;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t e = w & 0x000f000fu, o = w & 0x00f000f0u;
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&e));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&o));
    x[i] = fmaf(even, a.x, lo);
    x[i + 1] = fmaf(odd, b.x, lo);
    x[i + 4] = fmaf(even, a.y, lo);
    x[i + 5] = fmaf(odd, b.y, lo);
    w >>= 8;
  }
}

}  // namespace ra
