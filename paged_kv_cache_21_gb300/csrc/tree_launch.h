// paged_tree_attention: parameters and host entry points shared by its CUDA
// translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace pkv {

// The least range of a CTA, in pages: two chunks, so that a short context needs no
// second kernel's work on its parts (1 x 1024 tokens, 8 KV heads: 16.1 us with 4 pages,
// 14.6 with 8, 13.4 with 16, 15.7 with 32).
constexpr int kMinPages = 16;

// What a (sequence, KV head) costs a CTA beside its pages, in pages: a multiple of
// the least range, so that short contexts are cut at their pages.  (64 contexts of 16
// to 16384 tokens, by kernel for few, many rows: 219 us with 0, 48; 195 with 16, 48; 177
// with 32, 48; 172 with 32, 32; 172 with 48, 32; 331 for none and both least ranges 4.)
constexpr int kExtraPages = 32;

struct TreeParams {
    const uint16_t* q;          // bf16 [total][Hq][D]
    void* out;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const int32_t* bt;
    const int32_t* ctx;
    const int32_t* starts;
    const int32_t* parents;
    float* part_o;              // [CTAs][2][rows of a CTA][D]
    float2* part_ml;            // [CTAs][2][rows of a CTA]: (max in log2 units, sum)
    int4* meta;                 // [CTAs]: (sequence, KV head, partials, rows)
    int B, total, max_nodes, Hq, Hkv, G, max_blocks, num_blocks;
    uint32_t g_magic;           // ceil(2^32 / G), 0 for G == 1
    int nctas;                  // CTAs of a team
    int teams;
    int min_q;                  // least pages of a CTA's range
    int rows_above, rows_to;    // the sequences served: rows_above < n * G <= rows_to
    int tidy;                   // this kernel raises the table flags and zeroes empty sequences
    float sl2, v_scale;
    int out_f32;
    long long test_stall;
};

// Query rows per KV head up to which a sequence is served by the kernel for few rows.
// (32 x 8192 tokens, 4 heads per KV head, 36 and 64 rows: 168 and 172 us by that kernel,
// 235 and 238 by the other; E4M3: 152 and 157 against 198 and 207.)
constexpr int kSmallRows = 64;

// The kernel for few rows: rows (32 or 64) of its instantiation for the most
// rows a sequence may have there, and its launch (grid p.nctas).
int tree_small_rows(int rows);
cudaError_t tree_small_launch(const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, int D,
                              bool fp8, int rows, cudaStream_t st);
int tree_small_read_error(unsigned* flags, long long* detail);

}  // namespace pkv
