// Tensor maps over the paged caches, shared by the CUDA translation units of
// libpagedkv (paged_decode.cu builds and keeps them).
#pragma once

#include <cuda.h>

namespace pkv {

// The map of one cache viewed as [num_blocks * Hkv][16][D]: boxes of 16 token
// rows x 128 bytes (64 for E4M3 at head_dim 64) with the swizzle of that width.
int cache_tensor_map(CUtensorMap* map, const void* base, int D, bool fp8, int num_blocks,
                     int Hkv);

}  // namespace pkv
