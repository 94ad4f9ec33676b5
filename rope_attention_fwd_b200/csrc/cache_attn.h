// cache_attn.h -- launchers of the kernels behind rope_attn_cache_attn.
#pragma once
#include <cuda_runtime.h>

#include "serving.h"

namespace ra {

struct AttnArgs;

// bf16, few rows: sets a.tile for `rows`, the most rows of a sequence and kv head that a takes,
// and the number of blocks launched.
cudaError_t launch_cache_rows(AttnArgs& a, long long rows, int* blocks, cudaStream_t s);
// bf16, sequences of many rows: kChunkBlocks blocks, tiles of kChunkTile rows.
cudaError_t launch_cache_chunk(AttnArgs& a, cudaStream_t s);
}  // namespace ra
