// paged_latent_attention: parameters and host entry points shared by its CUDA
// translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace pkv {

struct LatentParams {
    uint16_t* out;              // bf16 [total][H][L]
    const uint16_t* cache;
    const int32_t* bt;
    const int32_t* ctx;
    const int32_t* starts;      // or null: node s is sequence s
    const int32_t* parents;
    float* part_o;              // [workers][2][rows of a tile][L]
    float2* part_ml;            // [workers][2][rows of a tile]: (max in log2 units, sum)
    int4* meta;                 // [workers]: (sequence, tile, partials, rows)
    int B, total, max_nodes, H, R, max_blocks, num_blocks;
    int workers;                // that share the pages out: CTAs, or pairs of them
    int tile_rows;
    uint32_t h_magic;           // ceil(2^32 / H), 0 for H == 1
    float sl2;
    long long test_stall;
};

// Rows (tokens times heads) that the largest sequence of a call may have to be served by
// the kernel for few rows.
constexpr int kLatentFew = 64;

cudaError_t latent_small_launch(const LatentParams& p, const void* q, const void* cache, int latent_dim, cudaStream_t st);
int latent_small_read_error(unsigned* flags, long long* detail);

// Rows of W bf16, as boxes of box_rows rows x box_cols 64-element columns with the
// 128-byte swizzle: column by column in shared memory.
int latent_column_map(CUtensorMap* map, const void* base, long long rows, int W, int cols, int box_rows, int box_cols);
// The same rows as they are, in boxes of 64 elements: of the one that starts at W - R, what
// lies behind the row is zeros.
int latent_row_map(CUtensorMap* map, const void* base, long long rows, int W, int box_rows);

}  // namespace pkv
