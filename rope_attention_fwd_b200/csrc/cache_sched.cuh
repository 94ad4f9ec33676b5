// cache_sched.cuh -- the device side of how the attention over the cache is cut (serving.h):
// every block of a launch of fixed size finds its run of steps from the lengths alone, walks
// the items in it, and leaves what the combine kernel needs.
#pragma once
#include <cuda_runtime.h>

#include <new>

#include "cache.cuh"
#include "serving.h"

namespace ra {

struct AttnArgs {
  CacheDims c;
  const uint8_t* cache;
  const int *table, *indptr, *kv_len;
  const void* q;
  int64_t q_n, q_h;          // strides of token and head (elements)
  int q_vec;                 // 16-byte loads fit
  void* o;                   // [T, Hq, d]
  float* lse;                // [T, Hq]
  PartDesc* desc;            // [gridDim.x]
  float* ml;                 // [2 gridDim.x][tile][2]
  float* acc;                // [2 gridDim.x][tile][d]
  uint32_t* err;
  uint64_t wait_ns;
  int tile, min_steps;       // rows of a tile; fewest steps of a block's run
  long long min_rows, max_rows;  // sequences of min_rows < rows <= max_rows are this kernel's
};

__device__ __forceinline__ SeqWork load_work(const AttnArgs& a, int b) {
  return seq_work(a.c, a.indptr[b], a.indptr[b + 1], a.kv_len[b], a.tile, a.min_rows,
                  a.max_rows);
}
struct WorkOf {  // the lengths in device memory, as Walk reads them
  const AttnArgs& a;  // a kernel's __grid_constant__ parameter
  __device__ SeqWork operator()(int b) const { return load_work(a, b); }
};

// Every thread of the block calls this; scratch: 8 bytes x (blockDim / 32 + 4) in shared
// memory.  Sequences are taken blockDim at a time: their totals are scanned once for the sum
// over the batch and, when there are more than blockDim, once more to find `begin`.
__device__ inline Run find_run(const AttnArgs& a, long long* scratch, int kid) {
  const int n = blockDim.x, warps = n / 32;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  long long total = 0, mine = 0, before = 0;
  auto chunk_scan = [&](int b0, long long& chunk) {  // mine, before: this thread's sequence
    const int b = b0 + (int)threadIdx.x;
    mine = b < a.c.B ? load_work(a, b).total : 0;
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    long long pre = 0;
    chunk = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) pre += scratch[w];
      chunk += scratch[w];
    }
    before = pre + x - mine;
    __syncthreads();
  };
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.c.B; b += n) {
      const int fault = sequence_fault(a.c, a.indptr[b], a.indptr[b + 1], a.kv_len[b]);
      if (fault) record_cache_fault(a.err, kid, fault, b);
    }
  Run r;
  if (a.c.B <= 32) {
    // a warp holds the whole batch: every warp finds the run for itself, nothing is shared
    mine = lane < a.c.B ? load_work(a, lane).total : 0;
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    total = __shfl_sync(0xffffffffu, x, 31);
    before = x - mine;
    r.per = steps_per_block(total, (int)gridDim.x, a.min_steps);
    r.whole = whole_steps(r.per, a.tile);
    r.begin = min(total, (long long)blockIdx.x * r.per);
    r.end = min(total, r.begin + r.per);
    const unsigned hit = __ballot_sync(
        0xffffffffu, mine > 0 && r.begin >= before && r.begin < before + mine);
    r.b = hit ? __ffs(hit) - 1 : 0;
    r.base = __shfl_sync(0xffffffffu, before, r.b);
    return r;
  }
  for (int b0 = 0; b0 < a.c.B; b0 += n) {
    long long chunk;
    chunk_scan(b0, chunk);
    total += chunk;
  }
  r.per = steps_per_block(total, (int)gridDim.x, a.min_steps);
  r.whole = whole_steps(r.per, a.tile);
  r.begin = min(total, (long long)blockIdx.x * r.per);
  r.end = min(total, r.begin + r.per);
  r.b = 0;
  r.base = 0;
  if (r.begin >= r.end) return r;
  long long off = 0;
  int* found = reinterpret_cast<int*>(scratch + warps);
  for (int b0 = 0; b0 < a.c.B; b0 += n) {
    long long chunk;
    if (a.c.B <= n) chunk = total;  // still in the registers
    else chunk_scan(b0, chunk);
    if (r.begin < off + chunk) {
      if (mine > 0 && r.begin >= off + before && r.begin < off + before + mine) {
        *found = b0 + (int)threadIdx.x;
        scratch[warps + 1] = off + before;
      }
      break;
    }
    off += chunk;
  }
  __syncthreads();
  r.b = *found;
  r.base = scratch[warps + 1];
  return r;
}

// A block's walk kept in shared memory and advanced by one thread, so that its state takes no
// registers of the others: seg[k % 2] is the block's k-th segment.
struct SharedWalk {
  Walk<WorkOf> walk;
  Segment seg[2];
  int more[2];

  __device__ void start(const AttnArgs& a, const Run& r) {
    new (&walk) Walk<WorkOf>(WorkOf{a}, r, a.c.B, a.c.Hkv);
    advance(0);
  }
  __device__ void advance(int k) { more[k % 2] = walk.next(seg[k % 2]); }
};

}  // namespace ra
