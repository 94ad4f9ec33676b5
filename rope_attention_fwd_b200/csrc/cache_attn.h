// cache_attn.h -- launchers of the kernels behind rope_attn_cache_attn.
#pragma once
#include <cuda_runtime.h>

#include "serving.h"

namespace ra {

struct AttnArgs;

cudaError_t launch_cache_combine(const AttnArgs& a, int blocks, int32_t dtype, int rows,
                                 cudaStream_t s);

}  // namespace ra
