// What the kernels of paged_latent_attention share (paged_latent.cu, for many query
// rows, and paged_latent_small.cu, for few): bounded waits, the cut of the work over
// workers, and the visibility of drafted tokens.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "latent_launch.h"
#include "paged_kv.h"
#include "tree_common.cuh"
#include "umma.cuh"

namespace pkv {

static __device__ DevErr g_latent_err;           // one per translation unit
static Launched g_launched;

namespace {

constexpr long long kWaitLimit = 1LL << 31;     // ~1 s of SM clocks
constexpr float kMaxLag = 8.f;                  // the reference maximum may lag by 2^8
constexpr int kCopiers = 6;                     // entries of M_ISSUED: of a CTA, and of the other CTA of a pair

// misc words: tensor-memory base; abort; chunks whose scores have been seen; the range: the
// pages before it (-1: no range) and before its end, its first page's sequence, tile, index
// and unit, that sequence's nodes, context and first node, the units of a share; the warps'
// units and pages while it is cut; how many chunks (queries: segments) each copying warp has
// arrived for
enum Misc {
    M_TMEM = 0, M_ABORT, M_SEEN, M_P0, M_P1, M_S0, M_T0, M_J0, M_B0, M_N0, M_L0, M_NODE0, M_Q, M_SUMS,
    M_ISSUED = M_SUMS + 2 * 16, M_WORDS = M_ISSUED + 2 * kCopiers
};

// Pages of this worker's range.
__device__ __forceinline__ int range_pages(const volatile int* misc)
{
    return misc[M_P0] < 0 ? 0 : misc[M_P1] - misc[M_P0];
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// a += the lower, b += the upper of two bf16.
__device__ __forceinline__ void add_bf16x2(float& a, float& b, uint32_t x)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "add.f32.bf16 %0, l, %0;\n\tadd.f32.bf16 %1, h, %1;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(x));
}

// Wait until the scores of chunk g have been seen: a count, not a barrier, whose phases one
// that lags behind could mistake for each other.
__device__ __forceinline__ bool wait_seen(int g, volatile int* misc)
{
    const long long t0 = clock64();
    while (misc[M_SEEN] <= g) {
        if (misc[M_ABORT] || clock64() - t0 > kWaitLimit) return false;
        __nanosleep(100);
    }
    return true;
}

// After a wait has run out, with every role at its end: the copies under way land.  Each phase of
// a barrier that counts copies has an arrival, with the bytes, of each of n copying warps, which
// have arrived for the first issued[0 .. n) of its chunks; where one of them has come further
// than another, the arrivals that are missing are made here, so that the phases end with the
// bytes.  (None is ahead by more than the ring: it waits there for products of what all have
// copied.)  One thread.
template <int kSlots, typename Bar>
__device__ __forceinline__ void land(const volatile int* issued, int n, Bar bar)
{
    int most = 0;
    for (int i = 0; i < n; ++i) most = max(most, issued[i]);
    for (int i = 0; i < n; ++i)
        for (int g = issued[i]; g < most; ++g) mbar_arrive(bar(g));
    for (int g = max(0, most - kSlots); g < most; ++g) mbar_wait_bounded(bar(g), (uint32_t)g / kSlots & 1u, kWaitLimit);
}

// Bring page `id` of the cache to L2: this lane's lines of it, one of 8 lanes'.
__device__ __forceinline__ void prefetch_page(const LatentParams& p, int id, int row_elems, int eighth)
{
    if (id < 0 || id >= p.num_blocks) return;
    const char* src = reinterpret_cast<const char*>(p.cache + (size_t)id * kBlock * row_elems);
    for (int x = eighth * 128; x < kBlock * row_elems * 2; x += 8 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + x));
}

// Sequences without a context get zeros for their nodes (threads 0 .. nthreads - 1 of the
// CTAs of the kernel that does it).
template <int LAT, typename SeqInfo>
__device__ __forceinline__ void zero_nodes(const LatentParams& p, const SeqInfo& q, int tid, int nthreads)
{
    uint4* o = reinterpret_cast<uint4*>(p.out + (size_t)q.t0 * p.H * LAT);
    for (size_t i = tid; i < (size_t)q.n * p.H * LAT / 8; i += nthreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------------- work

struct SeqInfo {
    int t0, n, L, base, nb, tiles;      // nb: pages, 0 without nodes; tiles of rows
};

// What follows from a sequence's nodes and context.
__device__ __forceinline__ void seq_work(const LatentParams& p, SeqInfo& q)
{
    q.base = q.L > q.n ? q.L - q.n : 0;
    const int rows = q.n * p.H;
    q.tiles = (rows + p.tile_rows - 1) / p.tile_rows;
    q.nb = q.n > 0 ? (q.L + kBlock - 1) / kBlock : 0;
}

__device__ __forceinline__ SeqInfo seq_info(const LatentParams& p, int s, bool flag)
{
    SeqInfo q;
    int bad = 0;
    int L = __ldg(p.ctx + s);
    if (!p.starts) {
        q.t0 = s;
        q.n = 1;
    } else if (!tree_span(p.starts, s, p.total, p.max_nodes, q.t0, q.n, bad) && flag) {
        raise_flag(&g_latent_err, KV_DEVERR_BAD_TREE, bad);
    }
    const int cap = p.max_blocks * kBlock;
    if (L < 0 || L > cap) {
        if (flag) raise_flag(&g_latent_err, KV_DEVERR_CONTEXT_TOO_LONG, L);
        L = L < 0 ? 0 : cap;
    }
    if (flag && L > 0 && L < q.n) raise_flag(&g_latent_err, KV_DEVERR_BAD_TREE, L);
    q.L = L;
    seq_work(p, q);
    return q;
}

// The segments of a worker's range: the pages [j, j + np) of one (sequence, tile) each.
// Every role walks the same list, in chunks of kPages pages.
template <int kPages>
struct Walk {
    int s, tile, j, rem, seg, np;
    SeqInfo q;
    __device__ __forceinline__ Walk(const LatentParams& p, const volatile int* misc)
    {
        s = misc[M_S0];
        tile = misc[M_T0];
        j = misc[M_J0];
        rem = range_pages(misc);
        seg = 0;
        np = 0;
        if (rem > 0) {
            q.t0 = misc[M_NODE0];
            q.n = misc[M_N0];
            q.L = misc[M_L0];
            seq_work(p, q);
            np = min(q.nb - j, rem);
        }
    }
    __device__ __forceinline__ bool more() const { return rem > 0; }
    __device__ __forceinline__ int chunks() const { return (np + kPages - 1) / kPages; }
    __device__ __forceinline__ int chunk_pages(int c) const { return min(kPages, np - c * kPages); }
    // does chunk c reach the drafted positions, or the context's end?
    __device__ __forceinline__ bool drafted(int c) const
    {
        return (j + c * kPages + chunk_pages(c)) * kBlock > q.base;
    }
    __device__ __forceinline__ bool whole() const { return j == 0 && np == q.nb; }
    __device__ __forceinline__ void next(const LatentParams& p)
    {
        rem -= np;
        ++seg;
        if (rem <= 0) return;
        j = 0;
        if (++tile == q.tiles) {
            tile = 0;
            do {
                if (++s >= p.B) {
                    rem = 0;
                    return;
                }
                q = seq_info(p, s, false);
            } while (q.nb == 0);
        }
        np = min(q.nb, rem);
    }
};

// This worker's range: the list of pages, by sequence and tile, is cut into equal shares of at
// least min_q units, where a page is a unit and each (sequence, tile) costs extra more before its
// first page.  One warp where its lanes have a sequence each; else the CTA's threads together
// (a warp alone: 113 us for 1024 sequences of 256 tokens and 16 heads; so 96).
template <int kThreads>
__device__ __forceinline__ void cut_work(const LatentParams& p, volatile int* misc, int min_q, int extra, int worker, bool flag, int tid)
{
    constexpr int kWarps = kThreads / 32;
    static_assert(kWarps <= 16, "misc words");
    const int lane = tid & 31, warp = tid >> 5;
    const bool alone = p.B <= 32;
    if (!alone || warp == 0) {
        SeqInfo q;
        int u, n, iu, in;                        // this thread's sequence's units and pages; with those before
        int units, pages;                        // of the sequences at hand
        auto take = [&](int b, bool raise) {
            u = n = 0;
            if (b + tid < p.B) {
                q = seq_info(p, b + tid, raise);
                u = q.nb > 0 ? (q.nb + extra) * q.tiles : 0;
                n = q.nb * q.tiles;
            }
            iu = u;
            in = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int tu = __shfl_up_sync(kFull, iu, o), tn = __shfl_up_sync(kFull, in, o);
                if (lane >= o) {
                    iu += tu;
                    in += tn;
                }
            }
            units = __shfl_sync(kFull, iu, 31);
            pages = __shfl_sync(kFull, in, 31);
            if (alone) {
                __syncwarp();
                return;
            }
            __syncthreads();                     // (the sums before have been read)
            if (lane == 0) {
                misc[M_SUMS + warp] = units;
                misc[M_SUMS + 16 + warp] = pages;
            }
            __syncthreads();
            units = pages = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int tu = misc[M_SUMS + w], tn = misc[M_SUMS + 16 + w];
                iu += w < warp ? tu : 0;
                in += w < warp ? tn : 0;
                units += tu;
                pages += tn;
            }
        };
        if (tid == 0) misc[M_P0] = -1;           // (take's barriers are between this and the range's)
        // (all units are less than 2^31: the host has checked)
        int total = 0, all = 0;
        for (int b = 0; b < p.B; b += kThreads) {
            take(b, flag);
            total += units;
            all += pages;
        }
        const int share = max(min_q, (int)(((uint32_t)total + (uint32_t)p.workers - 1u) / (uint32_t)p.workers));
        const int lo = (int)min((long long)worker * share, (long long)total);
        const int hi = (int)min((long long)lo + share, (long long)total);
        int units0 = 0, pages0 = 0;              // before the sequences at hand
        for (int b = 0; b < p.B; b += kThreads) {
            if (p.B > kThreads) take(b, false);
            // the first page at or behind the range's ends
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int off = (e == 0 ? lo : hi) - (units0 + iu - u);
                if (off < 0 || off >= u) continue;
                const int v = q.nb + extra, t = off / v, j = max(0, off - t * v - extra);
                const int before = pages0 + in - n + t * q.nb + j;
                misc[e == 0 ? M_P0 : M_P1] = before;
                if (e == 1) continue;
                misc[M_S0] = b + tid;
                misc[M_T0] = t;
                misc[M_J0] = j;
                misc[M_B0] = units0 + iu - u + t * v + extra + j;
                misc[M_N0] = q.n;
                misc[M_L0] = q.L;
                misc[M_NODE0] = q.t0;
            }
            units0 += units;
            pages0 += pages;
        }
        if (tid == 0) {
            misc[M_Q] = share;
            if (hi >= total) misc[M_P1] = all;
        }
    }
    __syncthreads();
}

// Node (within the sequence) of row r of its rows.
__device__ __forceinline__ int row_node(const LatentParams& p, int r)
{
    return p.h_magic ? (int)__umulhi((uint32_t)r, p.h_magic) : r;
}

// The nodes that node i sees, as bits; false for a padding node.
__device__ __forceinline__ bool seen_nodes(const LatentParams& p, int t0, int i, DevErr* e, uint32_t (&m)[4])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = 0u;
    if (!p.starts || !p.parents) {
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = i >= 32 * k + 31 ? ~0u : i >= 32 * k ? (2u << (i - 32 * k)) - 1u : 0u;
        return true;
    }
    for (int a = i; a >= 0;) {
        const int up = tree_parent(p.parents, t0, a, e);
        if (up == KV_TREE_PAD) return a != i;
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] |= (a >> 5) == k ? 1u << (a & 31) : 0u;
        a = up;
    }
    return true;
}

// Bits [at, at + 32) of a string of 128, zero outside it.
__device__ __forceinline__ uint32_t bits_at(const uint32_t (&m)[4], int at)
{
    if (at <= -32 || at >= 128) return 0u;
    auto word = [&](int k) { return k == 0 ? m[0] : k == 1 ? m[1] : k == 2 ? m[2] : k == 3 ? m[3] : 0u; };
    if (at < 0) return m[0] << -at;
    return __funnelshift_r(word(at >> 5), word((at >> 5) + 1), at & 31);
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

}  // namespace
}  // namespace pkv
