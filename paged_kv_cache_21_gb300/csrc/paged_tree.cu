// paged_tree_attention: attention of a tree of drafted tokens over a
// block-paged KV cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "device_common.cuh"
#include "internal.h"
#include "paged_kv.h"
#include "tree_common.cuh"

namespace pkv {

__device__ DevErr g_tree_err;

namespace {

struct TreeParams {
    const uint16_t* q;          // bf16 [total][Hq][D]
    void* out;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const int32_t* bt;
    const int32_t* ctx;
    const int32_t* starts;
    const int32_t* parents;
    int B, total, max_nodes, Hq, Hkv, G, max_blocks, num_blocks;
    float sl2, v_scale;
    int out_f32;
};

// One warp per (node, query head): lane l holds elements l, l + 32, ... of the
// query and of the accumulator; one key after the other.
template <int D, bool FP8>
__global__ void __launch_bounds__(128) paged_tree_simple_kernel(const TreeParams p)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int s = blockIdx.y;
    int t0, n, bad = 0;
    const bool span_ok = tree_span(p.starts, s, p.total, p.max_nodes, t0, n, bad);
    int L = __ldg(p.ctx + s);
    const int cap = p.max_blocks * kBlock;
    if (!span_ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_flag(&g_tree_err, KV_DEVERR_BAD_TREE, bad);
        return;
    }
    if (L < 0 || L > cap) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            raise_flag(&g_tree_err, KV_DEVERR_CONTEXT_TOO_LONG, L);
        L = L < 0 ? 0 : cap;
    }
    if (L > 0 && L < n && blockIdx.x == 0 && threadIdx.x == 0)
        raise_flag(&g_tree_err, KV_DEVERR_BAD_TREE, L);
    const int base = L > n ? L - n : 0;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= n * p.Hq) return;
    const int i = row / p.Hq, hq = row % p.Hq, h = hq / p.G;
    // ancestors of the node, itself among them
    uint32_t anc[4] = {0u, 0u, 0u, 0u};
    bool pad = false;
    for (int a = i; a >= 0;) {
        const int par = tree_parent(p.parents, t0, a, &g_tree_err);
        if (par == KV_TREE_PAD) {
            pad = a == i;
            break;
        }
        anc[a >> 5] |= 1u << (a & 31);
        a = par;
    }
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __uint_as_float((uint32_t)p.q[((size_t)(t0 + i) * p.Hq + hq) * D + lane + 32 * e]
                               << 16);
        o[e] = 0.f;
    }
    for (int j = 0; j < L && !pad; ++j) {
        const int a = j - base;
        if (a >= 0 && !((anc[a >> 5] >> (a & 31)) & 1)) continue;
        const int blk = __ldg(p.bt + (size_t)s * p.max_blocks + j / kBlock);
        if (blk < 0 || blk >= p.num_blocks) {
            raise_flag(&g_tree_err, KV_DEVERR_BLOCK_OUT_OF_RANGE, blk);
            continue;
        }
        const size_t at = (((size_t)blk * p.Hkv + h) * kBlock + j % kBlock) * D + lane;
        float k[E], v[E], x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (FP8) {
                const __half_raw hk = __nv_cvt_fp8_to_halfraw(p.k_cache[at + 32 * e], __NV_E4M3);
                const __half_raw hv = __nv_cvt_fp8_to_halfraw(p.v_cache[at + 32 * e], __NV_E4M3);
                k[e] = __half2float(hk);
                v[e] = __half2float(hv);
            } else {
                k[e] = __uint_as_float(
                    (uint32_t) reinterpret_cast<const uint16_t*>(p.k_cache)[at + 32 * e] << 16);
                v[e] = __uint_as_float(
                    (uint32_t) reinterpret_cast<const uint16_t*>(p.v_cache)[at + 32 * e] << 16);
            }
            x = fmaf(q[e], k[e], x);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(kFull, x, d);
        x *= p.sl2;
        const float mn = fmaxf(m, x);
        const float c = mn == -INFINITY ? 1.f : exp2f(m - mn);
        const float w = mn == -INFINITY ? 0.f : exp2f(x - mn);
        l = l * c + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + w * v[e];
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : p.v_scale / l;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const size_t at = ((size_t)(t0 + i) * p.Hq + hq) * D + lane + 32 * e;
        const float r = l == 0.f ? 0.f : o[e] * inv;
        if (p.out_f32)
            static_cast<float*>(p.out)[at] = r;
        else
            static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(r);
    }
}

int check_tree_shape(int num_seqs, int max_nodes, int Hq, int Hkv, int D, int kv_dtype)
{
    if (num_seqs < 0 || max_nodes < 1 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0)
        return KV_ERR_INVALID_ARG;
    if (max_nodes > KV_TREE_MAX_NODES) return KV_ERR_TOO_LARGE;
    if (Hq / Hkv > 128) return KV_ERR_UNSUPPORTED;
    if (D != 64 && D != 128) return KV_ERR_UNSUPPORTED;
    if (kv_dtype != KV_DTYPE_BF16 && kv_dtype != KV_DTYPE_FP8_E4M3) return KV_ERR_UNSUPPORTED;
    return KV_OK;
}

}  // namespace

int tree_read_error(unsigned* flags, long long* detail)
{
    DevErr e;
    if (cudaMemcpyFromSymbol(&e, g_tree_err, sizeof e) != cudaSuccess) return KV_ERR_CUDA;
    DevErr z = {0u, -1LL};
    if (cudaMemcpyToSymbol(g_tree_err, &z, sizeof z) != cudaSuccess) return KV_ERR_CUDA;
    *flags = e.flags;
    *detail = e.flags ? e.detail : -1;
    return KV_OK;
}

}  // namespace pkv

using namespace pkv;

extern "C" int paged_tree_workspace_bytes(int num_seqs, int max_nodes, int num_q_heads,
                                          int num_kv_heads, int head_dim, int kv_dtype,
                                          size_t* bytes)
{
    if (!bytes) return KV_ERR_INVALID_ARG;
    *bytes = 0;
    if (int rc = check_tree_shape(num_seqs, max_nodes, num_q_heads, num_kv_heads, head_dim,
                                  kv_dtype))
        return rc;
    *bytes = 256;
    return KV_OK;
}

extern "C" int paged_tree_attention(void* out, int out_dtype, const void* q, const void* k_cache,
                                    const void* v_cache, int kv_dtype, float k_scale,
                                    float v_scale, int num_blocks, const int32_t* block_tables,
                                    int max_blocks_per_seq, const int32_t* context_lens,
                                    const int32_t* node_starts, const int32_t* parents,
                                    int num_seqs, int total_nodes, int max_nodes,
                                    int num_q_heads, int num_kv_heads, int head_dim, float scale,
                                    void* workspace, size_t workspace_bytes, void* stream)
{
    if (int rc = check_tree_shape(num_seqs, max_nodes, num_q_heads, num_kv_heads, head_dim,
                                  kv_dtype))
        return rc;
    if (out_dtype != KV_DTYPE_BF16 && out_dtype != KV_DTYPE_F32) return KV_ERR_UNSUPPORTED;
    if (total_nodes < 0) return KV_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_nodes == 0) return KV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !node_starts ||
        !workspace)
        return KV_ERR_INVALID_ARG;
    if (num_blocks <= 0 || max_blocks_per_seq <= 0) return KV_ERR_INVALID_ARG;
    if ((((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)workspace |
          (uintptr_t)out) & 15) != 0)
        return KV_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return KV_ERR_INVALID_ARG;
    const bool fp8 = kv_dtype == KV_DTYPE_FP8_E4M3;
    if (fp8 && !(k_scale > 0.f && v_scale > 0.f && std::isfinite(k_scale) && std::isfinite(v_scale)))
        return KV_ERR_INVALID_ARG;
    size_t need = 0;
    if (int rc = paged_tree_workspace_bytes(num_seqs, max_nodes, num_q_heads, num_kv_heads,
                                            head_dim, kv_dtype, &need))
        return rc;
    if (workspace_bytes < need) return KV_ERR_INVALID_ARG;
    if ((long long)num_seqs * max_blocks_per_seq * num_kv_heads >= INT_MAX ||
        (long long)num_blocks * num_kv_heads >= INT_MAX ||
        (long long)max_blocks_per_seq * kBlock >= INT_MAX || num_seqs > 65535)
        return KV_ERR_UNSUPPORTED;
    TreeParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.out = out;
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.bt = block_tables;
    p.ctx = context_lens;
    p.starts = node_starts;
    p.parents = parents;
    p.B = num_seqs;
    p.total = total_nodes;
    p.max_nodes = max_nodes;
    p.Hq = num_q_heads;
    p.Hkv = num_kv_heads;
    p.G = num_q_heads / num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.sl2 = scale * 1.4426950408889634f * (fp8 ? k_scale : 1.f);
    p.v_scale = fp8 ? v_scale : 1.f;
    p.out_f32 = out_dtype == KV_DTYPE_F32;
    const dim3 grid((unsigned)((max_nodes * num_q_heads + 3) / 4), (unsigned)num_seqs);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (head_dim == 128) {
        if (fp8) paged_tree_simple_kernel<128, true><<<grid, 128, 0, st>>>(p);
        else paged_tree_simple_kernel<128, false><<<grid, 128, 0, st>>>(p);
    } else {
        if (fp8) paged_tree_simple_kernel<64, true><<<grid, 128, 0, st>>>(p);
        else paged_tree_simple_kernel<64, false><<<grid, 128, 0, st>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}
