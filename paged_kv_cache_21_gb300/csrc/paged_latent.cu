// paged_latent_attention: attention of one token, or a tree of drafted tokens, over a
// cache that holds one row of L + R elements a token for all query heads.
//
//     out[i][h] = sum_j softmax_j(scale * q[i][h] . c_j) c_j[0 .. L)
//
// One CTA per (node, head); its warps take the positions in turn, each with a running
// maximum and sum, and are joined at the end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "device_common.cuh"
#include "internal.h"
#include "paged_kv.h"
#include "tree_common.cuh"

namespace pkv {

__device__ DevErr g_latent_err;
static Launched g_launched;

namespace {

constexpr int kWarps = 4;
constexpr int kMaxL = 512;

struct LatentParams {
    const uint16_t* q;
    const uint16_t* cache;
    uint16_t* out;
    const int32_t* bt;
    const int32_t* ctx;
    const int32_t* starts;
    const int32_t* parents;
    int B, total, max_nodes, H, L, R, max_blocks, num_blocks;
    float sl2;
};

__global__ void __launch_bounds__(kWarps * 32) paged_latent_kernel(const LatentParams p)
{
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][kMaxL];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int node = blockIdx.x / p.H, h = blockIdx.x % p.H;
    pdl_wait();
    // the sequence of the node
    int s = -1, t0 = 0, n = 0;
    if (!p.starts) {
        s = t0 = node;
        n = 1;
    } else {
        for (int x = 0; x < p.B; ++x) {
            int bad = 0;
            if (!tree_span(p.starts, x, p.total, p.max_nodes, t0, n, bad)) {
                if (blockIdx.x == 0 && tid == 0) raise_flag(&g_latent_err, KV_DEVERR_BAD_TREE, bad);
                continue;
            }
            if (node >= t0 && node < t0 + n) {
                s = x;
                break;
            }
        }
    }
    if (s < 0) return;
    int L = __ldg(p.ctx + s);
    const int cap = p.max_blocks * kBlock, i = node - t0;
    const bool flag = tid == 0 && h == 0 && i == 0;
    if (L < 0 || L > cap) {
        if (flag) raise_flag(&g_latent_err, KV_DEVERR_CONTEXT_TOO_LONG, L);
        L = L < 0 ? 0 : cap;
    }
    if (flag && L > 0 && L < n) raise_flag(&g_latent_err, KV_DEVERR_BAD_TREE, L);
    const int base = L > n ? L - n : 0;
    // the nodes that this one sees, as bits
    uint32_t seen[4] = {0u, 0u, 0u, 0u};
    const int32_t* parents = p.starts ? p.parents : nullptr;
    bool pad = false;
    for (int a = i; a >= 0;) {
        const int up = tree_parent(parents, t0, a, h == 0 && tid == 0 ? &g_latent_err : nullptr);
        if (up == KV_TREE_PAD) {
            pad = a == i;
            break;
        }
        seen[a >> 5] |= 1u << (a & 31);
        a = up;
    }
    const int W = p.L + p.R, pieces = W / 8;
    const uint16_t* q = p.q + ((size_t)node * p.H + h) * W;
    float x[3][8], o[3][8];
    for (int k = 0; k < 3; ++k) {
        for (int e = 0; e < 8; ++e) x[k][e] = o[k][e] = 0.f;
        const int c = lane + 32 * k;
        if (c < pieces)
            for (int e = 0; e < 8; ++e) x[k][e] = __uint_as_float((uint32_t)q[c * 8 + e] << 16);
    }
    float m = -INFINITY, l = 0.f;
    for (int j = warp; j < L && !pad; j += kWarps) {
        if (j >= base && !((seen[(j - base) >> 5] >> ((j - base) & 31)) & 1u)) continue;
        const int blk = __ldg(p.bt + (size_t)s * p.max_blocks + j / kBlock);
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0) raise_flag(&g_latent_err, KV_DEVERR_BLOCK_OUT_OF_RANGE, blk);
            continue;
        }
        const uint16_t* row = p.cache + ((size_t)blk * kBlock + j % kBlock) * W;
        float v[3][8], dot = 0.f;
        for (int k = 0; k < 3; ++k) {
            const int c = lane + 32 * k;
            for (int e = 0; e < 8; ++e) v[k][e] = c < pieces ? __uint_as_float((uint32_t)row[c * 8 + e] << 16) : 0.f;
            if (c < pieces)
                for (int e = 0; e < 8; ++e) dot += x[k][e] * v[k][e];
        }
        for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(kFull, dot, d);
        dot *= p.sl2;
        const float top = fmaxf(m, dot);
        const float a = m == -INFINITY ? 0.f : exp2f(m - top), w = dot == -INFINITY ? 0.f : exp2f(dot - top);
        m = top;
        l = l * a + (dot != dot ? dot : w);
        for (int k = 0; k < 3; ++k)
            for (int e = 0; e < 8; ++e) o[k][e] = o[k][e] * a + (dot != dot ? dot : w) * v[k][e];
    }
    for (int k = 0; k < 3; ++k) {
        const int c = lane + 32 * k;
        if (c * 8 < p.L)
            for (int e = 0; e < 8; ++e) s_o[warp][c * 8 + e] = o[k][e];
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    for (int w = 0; w < kWarps; ++w) sum += s_m[w] == -INFINITY ? (s_l[w] != s_l[w] ? s_l[w] : 0.f) : s_l[w] * exp2f(s_m[w] - M);
    bool any = !pad && base > 0;
    for (int a = 0; a < n && !pad; ++a) any = any || (a < L && ((seen[a >> 5] >> (a & 31)) & 1u));
    for (int d = tid; d < p.L; d += kWarps * 32) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += s_m[w] == -INFINITY ? 0.f : s_o[w][d] * exp2f(s_m[w] - M);
        v = sum != 0.f ? v / sum : any ? __uint_as_float(0x7fffffffu) : 0.f;
        reinterpret_cast<__nv_bfloat16*>(p.out)[((size_t)node * p.H + h) * p.L + d] = __float2bfloat16_rn(v);
    }
}

int check_latent_shape(int num_seqs, int max_nodes, int H, int L, int R)
{
    if (num_seqs < 0 || max_nodes < 1 || H <= 0 || L <= 0 || R <= 0) return KV_ERR_INVALID_ARG;
    if (max_nodes > KV_TREE_MAX_NODES) return KV_ERR_TOO_LARGE;
    if (H > 128 || (L != 256 && L != 512) || (R != 32 && R != 64)) return KV_ERR_UNSUPPORTED;
    return KV_OK;
}

}  // namespace

int latent_read_error(unsigned* flags, long long* detail) { return g_launched.take_error(g_latent_err, flags, detail); }

}  // namespace pkv

using namespace pkv;

extern "C" int paged_latent_workspace_bytes(int num_seqs, int max_nodes, int num_q_heads, int latent_dim,
                                            int rope_dim, size_t* bytes)
{
    if (!bytes) return KV_ERR_INVALID_ARG;
    *bytes = 0;
    if (int rc = check_latent_shape(num_seqs, max_nodes, num_q_heads, latent_dim, rope_dim)) return rc;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KV_ERR_CUDA;
    *bytes = 256;
    return KV_OK;
}

extern "C" int paged_latent_attention(void* out, const void* q, const void* cache, int num_blocks,
                                      const int32_t* block_tables, int max_blocks_per_seq,
                                      const int32_t* context_lens, const int32_t* node_starts,
                                      const int32_t* parents, int num_seqs, int total_nodes, int max_nodes,
                                      int num_q_heads, int latent_dim, int rope_dim, float scale,
                                      void* workspace, size_t workspace_bytes, void* stream)
{
    if (int rc = check_latent_shape(num_seqs, max_nodes, num_q_heads, latent_dim, rope_dim)) return rc;
    if (total_nodes < 0 || (!node_starts && (total_nodes != num_seqs || max_nodes != 1))) return KV_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_nodes == 0) return KV_OK;
    if (!out || !q || !cache || !block_tables || !context_lens || !workspace) return KV_ERR_INVALID_ARG;
    if (num_blocks <= 0 || max_blocks_per_seq <= 0) return KV_ERR_INVALID_ARG;
    if ((((uintptr_t)q | (uintptr_t)cache | (uintptr_t)workspace | (uintptr_t)out) & 15) != 0)
        return KV_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return KV_ERR_INVALID_ARG;
    if ((long long)total_nodes * num_q_heads >= INT_MAX - 256 || (long long)num_blocks * kBlock >= INT_MAX - 256 ||
        (long long)max_blocks_per_seq * kBlock >= INT_MAX)
        return KV_ERR_UNSUPPORTED;
    if (workspace_bytes < 256) return KV_ERR_INVALID_ARG;
    LatentParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.cache = static_cast<const uint16_t*>(cache);
    p.out = static_cast<uint16_t*>(out);
    p.bt = block_tables;
    p.ctx = context_lens;
    p.starts = node_starts;
    p.parents = parents;
    p.B = num_seqs;
    p.total = total_nodes;
    p.max_nodes = max_nodes;
    p.H = num_q_heads;
    p.L = latent_dim;
    p.R = rope_dim;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.sl2 = scale * 1.4426950408889634f;
    g_launched.note();
    paged_latent_kernel<<<(unsigned)(total_nodes * num_q_heads), kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}
