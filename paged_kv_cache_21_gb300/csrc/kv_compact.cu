// kv_tree_compact: the K and V of the accepted nodes of each sequence's draft
// tree move together, in place, in the caches of all layers at once.
//
// Node path[i] at position base + path[i] goes to position base + i.  The path
// is strictly increasing, so path[i] >= i and the source of move m > i lies
// behind the destination of move i: done in ascending order by the thread that
// owns a 16-byte column of the vectors, no move reads what an earlier one has
// written, and a batch of moves may load everything before it stores anything.
//
// What bounds it: nothing but the moved bytes, read and written once, and for
// one sequence the chain launch -> tables -> data.  One launch covers every
// layer (the pointers travel as kernel parameters): a launch a layer would cost
// more than the moves.  Measured: 64 sequences x 32 layers, 38.8 MB: 10.6 us (5.7 at
// HBM's rate, the rest launch and tables: launch, lengths, paths, block ids and
// the first loads wait for each other); one sequence: 6.5 us, host time (1.5 on the device).
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "internal.h"
#include "paged_kv.h"
#include "tree_common.cuh"

namespace pkv {

__device__ DevErr g_compact_err;
static Launched g_launched;

namespace {

constexpr int kLayersPerLaunch = 128;    // 2 KB of kernel parameters
constexpr int kThreads = 256;
constexpr int kBatch = 8;                // moves whose loads are in flight at once

struct CompactParams {
    uint4* cache[2][kLayersPerLaunch];   // K and V caches of the launch's layers
    const int32_t* bt;                   // [B][max_blocks]
    const int32_t* ctx;                  // [B]
    const int32_t* starts;               // [B + 1]
    const int32_t* nodes;                // [B][max_nodes]
    const int32_t* lens;                 // [B]
    int max_blocks, max_nodes, num_blocks;
    int Hkv;
    int chunks;                          // 16-byte chunks of one head's vector
    int columns;                         // layers * 2 * Hkv * chunks
};

__global__ void __launch_bounds__(kThreads) kv_tree_compact_kernel(
    const __grid_constant__ CompactParams p)
{
    // (source, destination) slots of the sequence's moves
    __shared__ long long s_src[KV_TREE_MAX_NODES], s_dst[KV_TREE_MAX_NODES];
    __shared__ int s_moves;
    const int s = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    // (starts while the kernel before drains; lets the next one start at its end only,
    // since that may read the caches early)
    pdl_wait();
    if (tid < 32) {
        int t0, n, bad = s;
        const bool span_ok = tree_span(p.starts, s, INT32_MAX, p.max_nodes, t0, n, bad);
        const int L = __ldg(p.ctx + s);
        int m = __ldg(p.lens + s);
        const long long base = (long long)L - n;
        // (nothing is cached of a sequence without a context: a padded batch's idle row)
        if (L == 0) m = 0;
        // a path that is not strictly increasing within the tree moves nothing
        bool ok = span_ok && m >= 0 && m <= n && (base >= 0 || n == 0 || L == 0);
        if (!ok) m = 0;
        int node[KV_TREE_MAX_NODES / 32];
#pragma unroll
        for (int k = 0; k < KV_TREE_MAX_NODES / 32; ++k) {
            const int i = 32 * k + lane;
            node[k] = -1;
            if (i < m) {
                const int32_t* row = p.nodes + (size_t)s * p.max_nodes;
                node[k] = __ldg(row + i);
                const int before = i > 0 ? __ldg(row + i - 1) : -1;
                if (node[k] <= before || node[k] >= n) ok = false;
            }
        }
        ok = __all_sync(kFull, ok);
        if (lane == 0 && blockIdx.x == 0 && !ok) raise_flag(&g_compact_err, KV_DEVERR_BAD_TREE, bad);
        int moves = 0;
#pragma unroll
        for (int k = 0; k < KV_TREE_MAX_NODES / 32; ++k) {
            const int i = 32 * k + lane;
            bool move = ok && i < m && node[k] != i;
            long long src = 0, dst = 0;
            if (move) {
                const long long sp = base + node[k], dp = base + i;
                const int32_t* row = p.bt + (size_t)s * p.max_blocks;
                // a position behind the table's row has no block
                const int sb = sp / kBlock < p.max_blocks ? __ldg(row + sp / kBlock) : -1;
                const int db = dp / kBlock < p.max_blocks ? __ldg(row + dp / kBlock) : -1;
                if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
                    if (blockIdx.x == 0)
                        raise_flag(&g_compact_err, KV_DEVERR_BLOCK_OUT_OF_RANGE,
                                   sb < 0 || sb >= p.num_blocks ? sb : db);
                    move = false;
                }
                // in units of one token row of one head: block and offset in it
                src = (long long)sb * p.Hkv * kBlock + sp % kBlock;
                dst = (long long)db * p.Hkv * kBlock + dp % kBlock;
            }
            const unsigned who = __ballot_sync(kFull, move);
            if (move) {
                const int at = moves + __popc(who & ((1u << lane) - 1));
                s_src[at] = src;
                s_dst[at] = dst;
            }
            moves += __popc(who);
        }
        if (lane == 0) s_moves = moves;
    }
    __syncthreads();
    const int moves = s_moves;
    if (moves == 0) return;
    for (int col = blockIdx.x * kThreads + tid; col < p.columns; col += gridDim.x * kThreads) {
        const int c = col % p.chunks, r = col / p.chunks;
        const int h = r % p.Hkv, lt = r / p.Hkv;
        uint4* cache = p.cache[lt & 1][lt >> 1] + (size_t)h * kBlock * p.chunks + c;
        for (int i0 = 0; i0 < moves; i0 += kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (i0 + k < moves) v[k] = cache[s_src[i0 + k] * p.chunks];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (i0 + k < moves) cache[s_dst[i0 + k] * p.chunks] = v[k];
        }
    }
}

}  // namespace

// Do any two of the caches (n of K, then n of V, of `bytes` each) overlap?
// (All pairs: 2016 for 32 layers, in loops without branches.)
static bool overlap(void* const* k, void* const* v, int n, uint64_t bytes)
{
    uint64_t hit = 0;
    auto among = [&](uint64_t a, void* const* b, int m) {
        for (int j = 0; j < m; ++j) hit |= (uint64_t)(a - (uint64_t)b[j] + (bytes - 1) < 2 * bytes - 1);
    };
    for (int i = 0; i < n; ++i) {
        among((uint64_t)k[i], k, i);
        among((uint64_t)v[i], v, i);
        among((uint64_t)v[i], k, n);
    }
    return hit != 0;
}

int compact_read_error(unsigned* flags, long long* detail) { return g_launched.take_error(g_compact_err, flags, detail); }

}  // namespace pkv

using namespace pkv;

extern "C" int kv_tree_compact(void* const* k_caches, void* const* v_caches, int num_layers,
                               const int32_t* block_tables, int max_blocks_per_seq,
                               const int32_t* context_lens, const int32_t* node_starts,
                               const int32_t* accept_nodes, const int32_t* accept_lens,
                               int num_seqs, int max_nodes, int num_kv_heads, int head_dim,
                               int num_blocks, int kv_dtype, void* stream)
{
    if (num_layers < 0 || num_seqs < 0 || max_nodes < 1 || num_kv_heads <= 0 || head_dim <= 0 ||
        num_blocks <= 0 || max_blocks_per_seq <= 0)
        return KV_ERR_INVALID_ARG;
    if (max_nodes > KV_TREE_MAX_NODES) return KV_ERR_TOO_LARGE;
    if (kv_dtype != KV_DTYPE_BF16 && kv_dtype != KV_DTYPE_FP8_E4M3) return KV_ERR_UNSUPPORTED;
    const long long row_bytes = (long long)head_dim * (kv_dtype == KV_DTYPE_BF16 ? 2 : 1);
    if (row_bytes % 16 != 0) return KV_ERR_UNSUPPORTED;
    if (num_layers == 0 || num_seqs == 0) return KV_OK;
    if (!k_caches || !v_caches || !block_tables || !context_lens || !node_starts ||
        !accept_nodes || !accept_lens)
        return KV_ERR_INVALID_ARG;
    for (int l = 0; l < num_layers; ++l)
        if (!k_caches[l] || !v_caches[l] ||
            (((uintptr_t)k_caches[l] | (uintptr_t)v_caches[l]) & 15) != 0)
            return KV_ERR_INVALID_ARG;
    // (a move done twice could read what the first one has written)
    if (overlap(k_caches, v_caches, num_layers, (uint64_t)num_blocks * num_kv_heads * kBlock * row_bytes))
        return KV_ERR_INVALID_ARG;
    if (num_seqs > 65535) return KV_ERR_TOO_LARGE;      // one grid row per sequence
    const long long per_layer = 2LL * num_kv_heads * (row_bytes / 16);
    if (per_layer * kLayersPerLaunch > INT32_MAX / 2) return KV_ERR_UNSUPPORTED;
    CompactParams p;
    p.bt = block_tables;
    p.ctx = context_lens;
    p.starts = node_starts;
    p.nodes = accept_nodes;
    p.lens = accept_lens;
    p.max_blocks = max_blocks_per_seq;
    p.max_nodes = max_nodes;
    p.num_blocks = num_blocks;
    p.Hkv = num_kv_heads;
    p.chunks = (int)(row_bytes / 16);
    g_launched.note();
    for (int l0 = 0; l0 < num_layers; l0 += kLayersPerLaunch) {
        const int nl = num_layers - l0 < kLayersPerLaunch ? num_layers - l0 : kLayersPerLaunch;
        for (int l = 0; l < nl; ++l) {
            p.cache[0][l] = static_cast<uint4*>(k_caches[l0 + l]);
            p.cache[1][l] = static_cast<uint4*>(v_caches[l0 + l]);
        }
        p.columns = (int)(per_layer * nl);
        // no more CTAs than run at once, so that the tables are looked up in one wave
        const int want = (p.columns + kThreads - 1) / kThreads, room = 8 * num_sms_current() / num_seqs;
        const dim3 grid((unsigned)(room < 1 ? 1 : want < room ? want : room), (unsigned)num_seqs);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3(kThreads);
        cfg.stream = static_cast<cudaStream_t>(stream);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, kv_tree_compact_kernel, p) != cudaSuccess) return KV_ERR_CUDA;
    }
    return KV_OK;
}
