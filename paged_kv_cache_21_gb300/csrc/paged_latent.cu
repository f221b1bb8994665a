// paged_latent_attention: attention of one token, or a tree of drafted tokens, over a
// cache that holds one row of L + R elements a token for all query heads.  Here: calls
// with more than 64 query rows a sequence, the merge of partial results, and the host side.
//
//     out[i][h] = sum_j softmax_j(scale * q[i][h] . c_j) c_j[0 .. L)
//
// Row r of a sequence's n * H rows is head r % H of node r / H.  A pair of CTAs (a
// cluster of two SMs) takes a tile of 128 rows, 64 each, and goes over pages of the
// context in chunks of 128 tokens (8 pages), with the products on the tensor cores of
// both together (tcgen05.mma.cta_group::2, M = 128):
//     S = Q K^T   (128 rows x 128 tokens; each CTA holds its 64 rows of Q and its 64
//                 tokens of K),
//     O += P V    (128 rows x L; each CTA holds its 64 rows of P and its half of V's
//                 columns, 128 of each 256, over all 128 tokens).
//
// Why a pair: 128 rows x 512 columns of O in float32 fill one SM's tensor memory, with no
// room for S, and 128 rows of Q (147 KB) with a chunk (147 KB) its shared memory.  Split
// so, a CTA holds Q 74 KB, K 74 KB, V 66 KB, P 16 KB; O takes 256 of its 512 columns of
// tensor memory, two buffers of S 128.
//
// What bounds it (L = 512, R = 64).  A chunk's 147 KB take HBM 1.68 us to two SMs (6.7
// TB/s, 152 SMs), ~3300 clocks.  A chunk's 36 products of N 128 and 16 of N 256 with their
// commits take ~3010 clocks (measured; one of N 128 takes 53, 45 at least whatever its N,
// one of N 256 65).  In the loop a chunk takes ~3500: 94 % of HBM's rate.
//
// Where a call's time goes, by stamps of the pairs (means, us; one call by itself, caches cold;
// back to back 78.4, 88.3 and 187):
//                                        32 x 8192    32 x 2048 x 4 tokens    1024 x 256
//   to the first scores (of it the cut)   9.4 (1.6)         10.9 (1.9)         15.6 (4.6)
//   the loop, over all tiles              39.3 x 1.36       19.0 x 2.42        3.1 x 13.8
//   a tile's last weights to its products  1.0 x 1.36        1.4 x 2.42        3.5 x 13.8
//   its result written                     2.5 x 1.36        2.9 x 2.42        3.3 x 13.8
//   to the next tile's first weights       0.9 x 0.36        0.7 x 1.42        1.0 x 12.8
//   pairs end apart (mean to last)         4.6               4.7                7.5
//   to the merge, the merge                2.0, 7.2          2.0, 10.8          2.5, 5.9
// (128 heads; a pair's range holds 1.36, 2.42 and 13.8 tiles or parts of them in the mean.)
//
// How:
//  * Each byte of the cache is copied twice, as K to one CTA and as V to either, and shared
//    memory has room for one chunk: a group of K's columns is copied again as soon as its
//    products are done, by a warp of its own (one warp for all groups and one for V: 92.6
//    us for the four tokens; so 88.4).  To have the second copy, and the first, find
//    their bytes in L2, a warp prefetches pages a chunk ahead, line by line (kAheadChunks;
//    by bulk copies to L2, which wait behind the others in the copy unit: 95 us for 84.7
//    without).
//  * Warps: eight weigh (two threads and two halves of O's columns a row), three copy K (the
//    first also Q), two V, two issue the MMAs of both CTAs (scores; products), one prefetches.
//  * The warps that copy V clear what must not be multiplied (0 * inf): rows behind the
//    context, and infinities and NaN of drafted rows, which some node may not see; the
//    latter come back as NaN to the rows that see them when the result is written.
//  * The scores of chunk c + 1 are computed while chunk c is weighed.
//  * The reference maximum of a row moves only when a score is more than 2^8 above it; then,
//    seldom, O's columns and the sums are scaled.
//  * Pairs of CTAs get equal shares of all the (sequence, tile, page)s.  The parts of a
//    (sequence, tile) go to the workspace in an order that the lanes, which are rows, write
//    together (6.6 -> 3 us), and are joined by a second kernel.
//  * Arrivals at the other CTA's barriers have no cluster-wide release (arrive_remote).
//
// Weights are rounded to bfloat16, and so sum up: an output is off by at most 2^-8 of the
// weighted absolute values, as its own rounding is; a second part would double the products.
//
// Chunks of 256 tokens (N 256 for the scores: 2206 clocks for 128 tokens), with K through a
// ring of columns and V through one of pages, were slower (98 us against 89 then): each
// column's copy, barrier and commit is on its own, and the rings hold less ahead.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "cache_map.h"
#include "internal.h"
#include "latent_kernel.cuh"

namespace pkv {

namespace {

constexpr int kPages = 8;                       // pages of a chunk
constexpr int kRows = 64;                       // rows of a CTA
constexpr int kTile = 2 * kRows;                // rows of a pair
// Chunks that are brought to L2 ahead of their copies.  (32 x 8192 tokens, 128 heads: 79.3 us
// with 1, 82.0 with 2, 84.8 with 3, 84.5 without; ragged 64 contexts 63.4, 64.7, 66.5, 66.3; 32 x 2048 x
// 4 tokens, where tensor cores bound it, 87.9, 89.1, 90.5, 86.7.)
constexpr int kAheadChunks = 1;
constexpr int kMinPages = 16;                   // least range of a pair of CTAs
// What a (sequence, tile) costs beside its pages: its queries, pipeline and results.  (With 24, 32,
// 40: ragged 64 contexts 64.3, 63.4, 64.1 us; 32 x 8192 79.6, 79.3, 80.1; 32 x 2048 x 4 tokens 88.1,
// 87.9, 88.0.)
constexpr int kExtraPages = 32;
template <int LAT>
struct Geo {
    static constexpr int kCols = LAT / 64;               // 64-element columns of the latent part
    static constexpr int kGroups = kCols / 4;            // groups of K columns; the rotary part is one more
    static constexpr int kHalves = LAT / 256;            // products of N 256 for a page
    static constexpr int kSlots = LAT == 512 ? 1 : 2;    // chunks of K and of V in shared memory
    static constexpr int kWeighWarps = 8, kKWarp = 8, kVWarp = 11, kMmaWarp = 13;
    static constexpr int kThreads = 16 * 32;             // (a warp a group of K, a half of V; one idle)
    static constexpr int kQBytes = (kCols + 1) * kRows * 128;
    static constexpr int kGroupBytes = kRows * 4 * 128;  // 64 tokens x 4 columns
    static constexpr int kRopeBytes = kRows * 128;
    static constexpr int kKSlot = kGroups * kGroupBytes + kRopeBytes;
    static constexpr int kVPage = kHalves * 4096;        // [256-column block][2 columns][16 tokens][128 B]
    static constexpr int kVSlot = kPages * kVPage;
    static constexpr int kPBytes = 2 * kRows * 128;      // [64 tokens][64 rows][128 B]
    static constexpr int kQOff = 0;
    static constexpr int kKOff = kQOff + kQBytes;
    static constexpr int kVOff = kKOff + kSlots * kKSlot;
    static constexpr int kPOff = kVOff + kSlots * kVSlot;
    static constexpr int kBarOff = kPOff + kPBytes;
    // barriers; (L): the first CTA's is the one that counts
    static constexpr int kG1 = kGroups + 1;
    // (B_QFULL, B_KFULL, B_VREADY: an arrival of either CTA, with the bytes that it copies)
    static constexpr int B_QFULL = 0;                            // (L) Q of both CTAs has landed
    static constexpr int B_QFREE = B_QFULL + 1;                  // the segment's last scores are computed
    static constexpr int B_KFULL = B_QFREE + 1;                  // (L) + slot * kG1 + group: K of both CTAs
    static constexpr int B_KFREE = B_KFULL + kSlots * kG1;       // + slot * kG1 + group
    static constexpr int B_VREADY = B_KFREE + kSlots * kG1;      // (L) + slot * 2 + half of the chunk: V of both CTAs
    static constexpr int B_VFREE = B_VREADY + kSlots * 2;        // likewise: its products are done
    static constexpr int B_VFIX = B_VFREE + kSlots * 2;          // + half: it has to be cleared and has landed here
    static constexpr int B_SFULL = B_VFIX + 2;                   // + buffer: scores
    static constexpr int B_SFREE = B_SFULL + 2;                  // (L) + buffer: both have read them
    static constexpr int B_PFULL = B_SFREE + 2;                  // (L) weights of both CTAs
    static constexpr int B_OFREE = B_PFULL + 1;                  // (L) both have read the accumulators
    static constexpr int B_EPI = B_OFREE + 1;                    // + segment & 1: likewise, for the clearing warps
    static constexpr int B_END = B_EPI + 2;                      // + MMA warp
    static constexpr int B_STALL = B_END + 2;                    // nothing arrives (the test hook)
    static constexpr int kNumBars = B_STALL + 1;
    static constexpr int kMiscOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kBadOff = kMiscOff + (M_WORDS * 4 + 15) / 16 * 16;      // [2][CTA of the pair][half][4] words
    static constexpr int kRedOff = kBadOff + 128;                 // [4][64] floats: maxima, sums
    static constexpr int kEnd = kRedOff + 4 * kRows * 4;
    static constexpr int kSmem = kEnd;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static_assert(1 + kG1 + 2 <= kCopiers, "misc words");
    // tensor memory: two buffers of S, then O
    static constexpr uint32_t kColO = 128, kTmemCols = kColO + kHalves * 128 <= 256 ? 256 : 512;
};

// ---------------------------------------------------------------- pairs of CTAs

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// The same shared-memory address in CTA `rank` of the pair.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrive on a barrier of either CTA.  What the other CTA's threads or MMAs then rely on is in
// this CTA's own shared and tensor memory, complete by the proxy fence and the tcgen05 waits
// before; a release at cluster scope, which waits for all that the thread has under way, took
// ~1400 clocks a chunk.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// The same, with bytes that this CTA's copies are going to count there.
__device__ __forceinline__ void arrive_remote_expect(uint32_t cluster_bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void store_remote(uint32_t cluster_addr, uint32_t x)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(x) : "memory");
}

// Stores to the other CTA's shared memory are performed before what follows.
__device__ __forceinline__ void fence_cluster()
{
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

// Tiled copies whose bytes count on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma2_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t cluster_bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
        : "memory");
}

__device__ __forceinline__ void tma2_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t cluster_bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(cluster_bar)
        : "memory");
}

__device__ __forceinline__ void mma2(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// Arrive on this barrier of both CTAs when every MMA issued before has completed.
__device__ __forceinline__ void commit2(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void give_up(volatile int* misc)
{
    misc[M_ABORT] = 1;
    store_remote(map_rank(smem_u32(const_cast<int*>(misc) + M_ABORT), cluster_rank() ^ 1u), 1u);
    raise_flag(&g_latent_err, KV_DEVERR_PIPELINE_TIMEOUT, blockIdx.x);
}

// Bounded wait that also gives up when another role of the pair has given up.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* misc)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (misc[M_ABORT]) return false;
        if (clock64() - t0 > kWaitLimit) {
            give_up(misc);
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* misc)
{
    return __all_sync(kFull, wait_bar(bar, parity, misc));
}

// ------------------------------------------------------------------------ kernel

template <int LAT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Geo<LAT>::kThreads, 1)
paged_latent_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qr,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_kr,
                    const __grid_constant__ CUtensorMap tm_v, const LatentParams p)
{
    using G = Geo<LAT>;
    extern __shared__ __align__(1024) uint8_t gb[];
    const uint32_t sb = smem_u32(gb);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1;
    volatile int* misc = reinterpret_cast<volatile int*>(gb + G::kMiscOff);
    // (the swizzle wants the base that the launch gives where there is no static shared memory)
    if (sb & 1023u) {
        if (tid == 0) raise_flag(&g_latent_err, KV_DEVERR_PIPELINE_TIMEOUT, sb);
        return;
    }
    auto bar = [&](int i) -> uint32_t { return sb + (uint32_t)(G::kBarOff + 8 * i); };
    auto lead = [&](int i) -> uint32_t { return map_rank(bar(i), 0u); };
    // chunk g: its slot and the parity of its pass
    auto slot = [](int g) -> int { return (int)((uint32_t)g % G::kSlots); };
    auto pass = [](int g) -> uint32_t { return (uint32_t)g / G::kSlots & 1u; };
    // its products are done
    auto done = [&](int g) -> uint32_t { return bar(G::B_VFREE + slot(g) * 2 + 1); };
    // the first CTA is told how far copying warp i of this one has come: Q, groups of K, halves of V
    auto issued = [&](int i, int n) {
        store_remote(map_rank(sb + (uint32_t)(G::kMiscOff + 4 * (M_ISSUED + 2 * i + (int)rank)), 0u), (uint32_t)n);
    };

    if (tid == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        mbar_init(bar(G::B_QFULL), 2);
        mbar_init(bar(G::B_QFREE), 1);
        for (int i = 0; i < G::kSlots * G::kG1; ++i) {
            mbar_init(bar(G::B_KFULL + i), 2);
            mbar_init(bar(G::B_KFREE + i), 1);
        }
        for (int i = 0; i < G::kSlots * 2; ++i) {
            mbar_init(bar(G::B_VREADY + i), 2);
            mbar_init(bar(G::B_VFREE + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(G::B_SFULL + i), 1);
            mbar_init(bar(G::B_SFREE + i), 2 * G::kWeighWarps);
            mbar_init(bar(G::B_END + i), 1);
            mbar_init(bar(G::B_EPI + i), 2 * G::kWeighWarps);
        }
        mbar_init(bar(G::B_PFULL), 2 * G::kWeighWarps);
        mbar_init(bar(G::B_OFREE), 2 * G::kWeighWarps);
        for (int i = 0; i < 2; ++i) mbar_init(bar(G::B_VFIX + i), 1);
        mbar_init(bar(G::B_STALL), 1);
        misc[M_ABORT] = 0;
        misc[M_SEEN] = 0;
        fence_mbar_init();
    }
    // (all this while the kernel before drains)
    if (warp == G::kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         sb + G::kMiscOff + 4 * M_TMEM),
                     "r"(G::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    umma::fence_before_sync();
    cluster_sync();                      // the barriers of both CTAs are there
    umma::fence_after_sync();
    pdl_launch_dependents();
    pdl_wait();
    cut_work<G::kThreads>(p, misc, kMinPages, kExtraPages, pair, blockIdx.x == 0, tid);
    const uint32_t tmem = (uint32_t)misc[M_TMEM];

    if (warp >= G::kKWarp && warp < G::kKWarp + G::kG1) {
        // ------------------------- Q and K: a warp for each group of K's columns
        const int k = warp - G::kKWarp;
        const bool rope = k == G::kGroups;
        int g = 0, queries = 0;
        bool ok = true;
        for (Walk<kPages> w(p, misc); ok && w.more(); w.next(p)) {
            if (k == 0 && w.seg > 0) ok = wait_warp(bar(G::B_QFREE), (uint32_t)((w.seg - 1) & 1), misc);
            if (!ok) break;
            if (k == 0 && lane == 0) {
                const int row = w.q.t0 * p.H + w.tile * kTile + (int)rank * kRows;
                const uint32_t qf = lead(G::B_QFULL);
                arrive_remote_expect(qf, (uint32_t)G::kQBytes);
#pragma unroll
                for (int x = 0; x < G::kGroups; ++x)
                    tma2_load_3d(sb + (uint32_t)(G::kQOff + x * 4 * kRows * 128), &tm_q, 0, row, 4 * x, qf);
                tma2_load_2d(sb + (uint32_t)(G::kQOff + G::kCols * kRows * 128), &tm_qr, LAT, row, qf);
            }
            ++queries;
            const int32_t* row = p.bt + (size_t)w.s * p.max_blocks + w.j;
            const int nc = w.chunks();
            int ids = lane < w.np ? __ldg(row + lane) : -1;           // pages 0..31 of the segment
            int ahead = 32 + lane < w.np ? __ldg(row + 32 + lane) : -1;
            for (int c = 0; ok && c < nc; ++c, ++g) {
                if (c > 0 && (c & 3) == 0) {
                    ids = ahead;
                    const int at = (c + 4) * kPages + lane;
                    ahead = at < w.np ? __ldg(row + at) : -1;
                }
                // lanes 0..7: the chunk's pages; this CTA's four go by 8 token rows
                const int id8 = __shfl_sync(kFull, ids, (c & 3) * kPages + (lane & 7));
                const bool in = lane < w.chunk_pages(c) && lane < kPages;
                const bool valid = in && id8 >= 0 && id8 < p.num_blocks;
                if (in && !valid && rank == 0 && k == 0) raise_flag(&g_latent_err, KV_DEVERR_BLOCK_OUT_OF_RANGE, id8);
                const unsigned all = __ballot_sync(kFull, valid);
                const int mypage = 4 * (int)rank + ((lane & 7) >> 1);
                const int id = __shfl_sync(kFull, ids, (c & 3) * kPages + mypage);
                const bool mine = lane < 8 && ((all >> mypage) & 1u);
                const int n = __popc(__ballot_sync(kFull, mine)), sl = slot(g), b = sl * G::kG1 + k;
                if (g >= G::kSlots && !wait_warp(bar(G::B_KFREE + b), pass(g) ^ 1u, misc)) {
                    ok = false;
                    break;
                }
                const uint32_t kb = sb + (uint32_t)(G::kKOff + sl * G::kKSlot);
                const uint32_t kf = lead(G::B_KFULL + b);
                if (lane == 0) arrive_remote_expect(kf, (uint32_t)(n * (rope ? 1024 : 4096)));
                __syncwarp();
                if (!rope) {
                    if (mine)
                        tma2_load_3d(kb + (uint32_t)(k * G::kGroupBytes + lane * 4096), &tm_k, 0,
                                     id * kBlock + 8 * (lane & 1), 4 * k, kf);
                } else if (mine && !(lane & 1)) {
                    tma2_load_2d(kb + (uint32_t)(G::kGroups * G::kGroupBytes + (lane >> 1) * 2048), &tm_kr, LAT,
                                 id * kBlock, kf);
                }
            }
        }
        if (lane == 0) {
            issued(1 + k, g);
            if (k == 0) issued(0, queries);
        }
        __syncwarp();
    } else if (warp == G::kVWarp || warp == G::kVWarp + 1) {
        // ------------- V, a warp for each half of a chunk; and what of it must not be multiplied: rows behind the context, and
        // infinities and NaN of drafted rows
        const int h = warp - G::kVWarp;
        int g = 0, fixes = 0;
        bool ok = true;
        for (Walk<kPages> w(p, misc); ok && w.more(); w.next(p)) {
            const int32_t* row = p.bt + (size_t)w.s * p.max_blocks + w.j;
            const int nc = w.chunks(), buf = w.seg & 1;
            // the notes of what is cleared were last read two segments ago
            if (w.seg >= 2) ok = wait_warp(bar(G::B_EPI + buf), (uint32_t)(((w.seg - 2) >> 1) & 1), misc);
            if (!ok) break;
            uint32_t bad[4] = {0u, 0u, 0u, 0u};          // drafted rows where something was cleared
            int ids = lane < w.np ? __ldg(row + lane) : -1;
            int ahead = 32 + lane < w.np ? __ldg(row + 32 + lane) : -1;
            for (int c = 0; ok && c < nc; ++c, ++g) {
                if (c > 0 && (c & 3) == 0) {
                    ids = ahead;
                    const int at = (c + 4) * kPages + lane;
                    ahead = at < w.np ? __ldg(row + at) : -1;
                }
                const int sl = slot(g);
                const bool fix = w.drafted(c);
                // lanes 0 .. 4 * halves - 1: page and 256-column block
                const int page = 4 * h + lane / G::kHalves % 4, t = lane % G::kHalves;
                const int id = __shfl_sync(kFull, ids, (c & 3) * kPages + page);
                const bool mine = lane < 4 * G::kHalves && page < w.chunk_pages(c) && id >= 0 && id < p.num_blocks;
                const int n = __popc(__ballot_sync(kFull, mine));
                const int b = sl * 2 + h;
                if (g >= G::kSlots && !wait_warp(bar(G::B_VFREE + b), pass(g) ^ 1u, misc)) {
                    ok = false;
                    break;
                }
                const uint32_t ready = lead(G::B_VREADY + b), full = fix ? bar(G::B_VFIX + h) : ready;
                if (lane == 0) {
                    if (fix) mbar_arrive_expect_tx(full, (uint32_t)(n * 4096));
                    else arrive_remote_expect(ready, (uint32_t)(n * 4096));
                }
                __syncwarp();
                if (mine)
                    tma2_load_3d(sb + (uint32_t)(G::kVOff + sl * G::kVSlot + page * G::kVPage + t * 4096), &tm_v, 0,
                                 id * kBlock, 4 * t + 2 * (int)rank, full);
                if (!fix) continue;
                // (they are this warp's copies alone, which land whatever the other roles do)
                if (!__all_sync(kFull, mbar_wait_bounded(full, (uint32_t)(fixes++ & 1), kWaitLimit))) {
                    if (lane == 0) give_up(misc);
                    ok = false;
                    break;
                }
                const int p0 = (w.j + c * kPages) * kBlock;
                const int lo = max(64 * h, w.q.base - p0), hi = min(64 * (h + 1), w.chunk_pages(c) * kBlock);
                // a row's 16-byte pieces, 16 of each 256-column block
                for (int r = lo; r < hi; ++r) {
                    const bool tail = p0 + r >= w.q.L;
                    for (int x = lane; x < 16 * G::kHalves; x += 32) {
                        const int tt = x >> 4, col = (x >> 3) & 1, ch = x & 7, rr = r & 15;
                        const uint32_t at = sb + (uint32_t)(G::kVOff + sl * G::kVSlot + (r >> 4) * G::kVPage +
                                                            tt * 4096 + col * 2048 + rr * 128 + ((ch ^ (rr & 7)) * 16));
                        uint32_t v[4] = {0u, 0u, 0u, 0u}, any = 0u;
                        if (!tail) {
                            lds128(v, at);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t m = __vcmpeq2(v[k] & 0x7f807f80u, 0x7f807f80u);
                                v[k] &= ~m;
                                any |= m;
                            }
                        }
                        if (tail || any) sts128(at, make_uint4(v[0], v[1], v[2], v[3]));
                        const int a = p0 + r - w.q.base;
#pragma unroll
                        for (int k = 0; k < 4; ++k) bad[k] |= any && (a >> 5) == k ? 1u << (a & 31) : 0u;
                    }
                }
                fence_proxy_async_smem();
                // both CTAs' rows have all columns, so both are told
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    bad[k] = __reduce_or_sync(kFull, bad[k]);
                    if (lane < 2) {
                        const uint32_t at = sb + (uint32_t)(G::kBadOff + (((buf * 2 + (int)rank) * 2 + h) * 4 + k) * 4);
                        store_remote(map_rank(at, (uint32_t)lane), bad[k]);
                    }
                }
                fence_cluster();
                __syncwarp();
                if (lane == 0) arrive_remote(ready);
            }
        }
        if (lane == 0) issued(1 + G::kG1 + h, g);
        __syncwarp();
    } else if (warp == G::kMmaWarp) {
        // ---------------------------------------------------------------- scores
        if (rank == 0 && lane == 0) {
            const uint64_t qdesc = umma::smem_desc_sw128(sb + G::kQOff, 16, 1024);
            const uint64_t kdesc = umma::smem_desc_sw128(sb + G::kKOff, 16, 4096);
            const uint64_t rdesc = umma::smem_desc_sw128(sb + G::kKOff + G::kGroups * G::kGroupBytes, 16, 1024);
            constexpr uint32_t idesc = umma::idesc_bf16_f32(128, 128, false, false);
            bool ok = true;
            if (p.test_stall > 0 && range_pages(misc) > 0 && !mbar_wait_bounded(bar(G::B_STALL), 0u, p.test_stall)) {
                give_up(misc);
                ok = false;
            }
            int g = 0;
            for (Walk<kPages> w(p, misc); ok && w.more(); w.next(p)) {
                const int nc = w.chunks();
                ok = wait_bar(bar(G::B_QFULL), (uint32_t)(w.seg & 1), misc);
                for (int c = 0; ok && c < nc; ++c, ++g) {
                    // the buffer was read for chunk g - 2
                    if (g >= 2) ok = wait_bar(bar(G::B_SFREE + (g & 1)), (uint32_t)((g >> 1) - 1) & 1u, misc);
                    const int sl = slot(g);
                    const uint32_t d = tmem + (uint32_t)(64 * (g & 1));
                    const uint64_t ks = (uint64_t)((sl * G::kKSlot) >> 4);
#pragma unroll
                    for (int k = 0; k <= G::kGroups; ++k) {
                        const int b = sl * G::kG1 + k;
                        ok = ok && wait_bar(bar(G::B_KFULL + b), pass(g), misc);
                        if (!ok) break;
                        umma::fence_after_sync();
                        if (k < G::kGroups) {
#pragma unroll
                            for (int kk = 0; kk < 16; ++kk)
                                mma2(d, qdesc + (uint64_t)(((k * 4 + (kk >> 2)) * kRows * 128 + (kk & 3) * 32) >> 4),
                                     kdesc + ks + (uint64_t)((k * G::kGroupBytes + (kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                                     idesc, k + kk > 0);
                        } else {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma2(d, qdesc + (uint64_t)((G::kCols * kRows * 128 + kk * 32) >> 4),
                                     rdesc + ks + (uint64_t)((kk * 32) >> 4), idesc, true);
                        }
                        commit2(bar(G::B_KFREE + b));
                    }
                    if (!ok) break;
                    commit2(bar(G::B_SFULL + (g & 1)));
                    if (c + 1 == nc) commit2(bar(G::B_QFREE));
                }
            }
            // every MMA issued by this thread is complete before the pair ends
            commit2(bar(G::B_END));
            mbar_wait_bounded(bar(G::B_END), 0u, kWaitLimit);
        }
        __syncwarp();
    } else if (warp == G::kMmaWarp + 1) {
        // -------------------------------------------------------------- products
        if (rank == 0 && lane == 0) {
            const uint64_t pdesc = umma::smem_desc_sw128(sb + G::kPOff, 16, 1024);
            const uint64_t vdesc = umma::smem_desc_sw128(sb + G::kVOff, 2048, 1024);
            constexpr uint32_t idesc = umma::idesc_bf16_f32(128, 256, false, true);
            bool ok = true;
            int g = 0;
            for (Walk<kPages> w(p, misc); ok && w.more(); w.next(p)) {
                const int nc = w.chunks();
                // the accumulators of the segment before have been read
                if (w.seg > 0) ok = wait_bar(bar(G::B_OFREE), (uint32_t)((w.seg - 1) & 1), misc);
                for (int c = 0; ok && c < nc; ++c, ++g) {
                    const int sl = slot(g), np = w.chunk_pages(c);
                    ok = wait_bar(bar(G::B_PFULL), (uint32_t)(g & 1), misc);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int b = sl * 2 + h;
                        ok = ok && wait_bar(bar(G::B_VREADY + b), pass(g), misc);
                        if (!ok) break;
                        umma::fence_after_sync();
                        const int to = min(np, 4 * h + 4);
                        for (int k = 4 * h; k < to; ++k)
#pragma unroll
                            for (int t = 0; t < G::kHalves; ++t)
                                mma2(tmem + G::kColO + (uint32_t)(128 * t),
                                     pdesc + (uint64_t)(((k >> 2) * kRows * 128 + (k & 3) * 32) >> 4),
                                     vdesc + (uint64_t)((sl * G::kVSlot + k * G::kVPage + t * 4096) >> 4), idesc, c + k > 0);
                        commit2(bar(G::B_VFREE + b));
                    }
                }
            }
            commit2(bar(G::B_END + 1));
            mbar_wait_bounded(bar(G::B_END + 1), 0u, kWaitLimit);
        }
        __syncwarp();
    } else if (warp == G::kMmaWarp + 2) {
        // --------- this CTA's pages of the chunks to come, to L2, a few chunks ahead of the copies
        int g = 0;
        bool ok = true;
        for (Walk<kPages> w(p, misc); ok && w.more(); w.next(p)) {
            const int32_t* row = p.bt + (size_t)w.s * p.max_blocks + w.j;
            const int nc = w.chunks();
            // (the first chunks are copied at once)
            for (int a = 1; ok && a < nc; ++a) {
                if (a > kAheadChunks) ok = __all_sync(kFull, wait_seen(g + a - kAheadChunks - 1, misc));
                const int page = a * kPages + 4 * (int)rank + (lane & 3);
                if (ok) prefetch_page(p, page < w.np ? __ldg(row + page) : -1, LAT + p.R, lane >> 2);
            }
            g += nc;
        }
        // (the commits arrive in both CTAs, and the MMA threads see those of the first: the second's
        // are waited for here, off the path of the pair's end)
        if (rank == 1 && lane < 2) mbar_wait_bounded(bar(G::B_END + lane), 0u, kWaitLimit);
        __syncwarp();
    } else if (warp < G::kWeighWarps) {
        // --------------------------------------------------- weights and output
        const int wq = warp & 3, wg = warp >> 2;
        const int row = (wq & 1) * 32 + lane;    // of the CTA's 64
        const int kh = wq >> 1;                  // half of the chunk's tokens, and of an O block's columns
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        float* red = reinterpret_cast<float*>(gb + G::kRedOff);
        const volatile uint32_t* badw = reinterpret_cast<const volatile uint32_t*>(gb + G::kBadOff);
        // sequences without a context: zeros for their nodes
        for (int s = blockIdx.x; s < p.B; s += gridDim.x) {
            const SeqInfo q = seq_info(p, s, false);
            if (q.L == 0 && q.n > 0) zero_nodes<LAT>(p, q, tid, G::kWeighWarps * 32);
        }
        if (rank == 0 && tid == 0) p.meta[pair] = make_int4(0, 0, 0, 0);
        int g0 = 0, flat = misc[M_B0];
        bool ok = true;
        // The CTA's eight warps meet: is `x` true anywhere?  Every warp comes to every
        // meeting, also one whose waits have run out, which the others learn there.
        auto meet = [&](bool x) -> bool {
            int r;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                "barrier.cta.red.or.pred q, 1, 256, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
                : "=r"(r)
                : "r"(x ? 1 : 0)
                : "memory");
            return r != 0;
        };
        for (Walk<kPages> w(p, misc); ok && w.more(); w.next(p)) {
            const int seg = w.seg, buf = seg & 1, nc = w.chunks(), rows = w.q.n * p.H;
            const int r = w.tile * kTile + (int)rank * kRows + row;       // of the sequence's rows
            uint32_t seen[4];
            bool live = r < rows;
            {
                const int i = live ? row_node(p, r) : 0;
                // (a node's entry is read by the thread of its first head here, for one flag)
                live = seen_nodes(p, w.q.t0, i, w.j == 0 && live ? &g_latent_err : nullptr, seen) && live;
            }
            const bool warp_live = __any_sync(kFull, live);
            const bool cta_live = w.tile * kTile + (int)rank * kRows < rows;
            float ref = -INFINITY, nref = live ? 0.f : -INFINITY, l[4] = {0.f, 0.f, 0.f, 0.f};
            bool pending = true;                 // a row has no reference yet
            for (int c = 0; c < nc; ++c) {
                const int g = g0 + c;
                ok = __all_sync(kFull, ok && wait_bar(bar(G::B_SFULL + (g & 1)), (uint32_t)((g >> 1) & 1), misc));
                if (tid == 0) misc[M_SEEN] = g + 1;
                umma::fence_after_sync();
                if (!cta_live) {                 // nothing here weighs anything
                    // (an arrival before the last chunk's weights are used would count for them)
                    if (g > 0) ok = __all_sync(kFull, ok && wait_bar(done(g - 1), pass(g - 1), misc));
                    umma::fence_before_sync();
                    __syncwarp();
                    if (ok && lane == 0) {
                        arrive_remote(lead(G::B_SFREE + (g & 1)));
                        arrive_remote(lead(G::B_PFULL));
                    }
                    continue;
                }
                float t[32];
                uint32_t vis = ~0u;
                const int np = w.chunk_pages(c), k0 = kh * 64 + wg * 32;  // this thread's first token
                const bool masked = w.drafted(c) || np < kPages;
                float most = -INFINITY;
                if (warp_live) {
                    umma::tmem_ld32(lanes + (uint32_t)(64 * (g & 1) + 32 * wg), *reinterpret_cast<uint32_t(*)[32]>(&t[0]));
                    umma::tmem_wait_ld();
                }
                umma::fence_before_sync();
                __syncwarp();
                if (ok && lane == 0) arrive_remote(lead(G::B_SFREE + (g & 1)));
                if (warp_live) {
                    // (the product rounded before the sum: the reference is such a product, and a
                    // fused remainder would grow with it)
                    const u64 f = pack2(p.sl2, p.sl2);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) unpack2(mul2(pack2(t[k], t[k + 1]), f), t[k], t[k + 1]);
                    if (masked) {
                        const int pos = (w.j + c * kPages) * kBlock + k0;
                        vis = (low_bits(w.q.base - pos) | bits_at(seen, pos - w.q.base)) & low_bits(min(w.q.L - pos, np * kBlock - k0));
#pragma unroll
                        for (int k = 0; k < 32; ++k) t[k] = (vis >> k) & 1u ? t[k] : -INFINITY;
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 32; k += 2) mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], t[k], t[k + 1]);
                    most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) + nref;
                }
                // does any row's reference lag too far behind, or has a wait run out?
                if (meet(!ok || most > kMaxLag || pending)) {
                    if (meet(!ok)) {
                        ok = false;
                        break;
                    }
                    // ---- new references: the largest score of each row in the chunk
                    float top = -INFINITY;
                    if (warp_live) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) top = max_nan(top, t[k]);
                    }
                    red[(wg * 2 + kh) * kRows + row] = top;
                    meet(false);
                    top = max_nan(max_nan(red[row], red[kRows + row]), max_nan(red[2 * kRows + row], red[3 * kRows + row]));
                    // a row whose first scores hold NaN is NaN whatever its reference: 0
                    if (ref == -INFINITY && top != top) top = 0.f;
                    float a = 1.f;
                    if (live && (ref == -INFINITY ? top > -INFINITY : top > ref + kMaxLag)) {
                        a = ref == -INFINITY ? 0.f : ex2(ref - top);
                        ref = top;
                        nref = -top;
                    }
                    // what has been accumulated follows, once the products under way are done
                    const bool moved = meet(a != 1.f) && c > 0;
                    if (moved) ok = wait_warp(done(g - 1), pass(g - 1), misc);
                    pending = meet(live && ref == -INFINITY);
                    if (meet(!ok)) {
                        ok = false;
                        break;
                    }
                    if (moved) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) l[k] *= a;
                        umma::fence_after_sync();
#pragma unroll 1
                        for (int c0 = 0; c0 < G::kHalves * 64; c0 += 16) {
                            const uint32_t at = lanes + G::kColO + (uint32_t)(wg * G::kHalves * 64 + c0);
                            uint32_t o[16];
                            umma::tmem_ld16(at, o);
                            umma::tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                            umma::tmem_st16(at, o);
                        }
                        umma::tmem_wait_st();
                    }
                }
                // ---- the weights
                uint32_t hi[16];
                if (warp_live) {
                    const u64 n2 = pack2(nref, nref);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float a, b;
                        unpack2(add2(pack2(t[k], t[k + 1]), n2), a, b);
                        hi[k / 2] = pack_bf16x2(ex2(a), ex2(b));
                        add_bf16x2(l[k & 2], l[(k & 2) + 1], hi[k / 2]);
                    }
                }
                // the buffer of P: the products of the chunk before are done.  (A wait that
                // runs out is told at the next meeting; nothing is written then.)
                if (g > 0) ok = __all_sync(kFull, ok && wait_bar(done(g - 1), pass(g - 1), misc));
                if (ok && warp_live) {
                    const uint32_t pb = sb + (uint32_t)(G::kPOff + kh * kRows * 128 + row * 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sts128(pb + (uint32_t)(((wg * 4 + k) ^ (row & 7)) * 16),
                               make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]));
                }
                fence_proxy_async_smem();
                umma::fence_before_sync();
                __syncwarp();
                if (ok && lane == 0) arrive_remote(lead(G::B_PFULL));
            }
            // the warps go on together, or not at all
            if (meet(!ok)) ok = false;
            if (!ok) break;
            // ---- the segment's result
            ok = wait_warp(done(g0 + nc - 1), pass(g0 + nc - 1), misc);
            umma::fence_after_sync();
            red[(wg * 2 + kh) * kRows + row] = (l[0] + l[1]) + (l[2] + l[3]);
            if (meet(!ok)) ok = false;
            if (!ok) break;
            const float sum = (red[row] + red[kRows + row]) + (red[2 * kRows + row] + red[3 * kRows + row]);
            const bool whole = w.whole(), in = r < rows;
            const size_t prow = ((size_t)pair * 2 + (w.j == 0 ? 1 : 0)) * kTile + rank * kRows + row;
            float z = 1.f;
            if (whole) {
                bool any = w.q.base > 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) any = any || (seen[k] & low_bits(w.q.L - 32 * k)) != 0u;
                // (a row that sees something and weighs nothing had scores of -inf alone)
                z = live && sum != 0.f ? 1.f / sum : live && any ? __uint_as_float(0x7fffffffu) : 0.f;
            } else if (in && wg == 0 && kh == 0) {
                p.part_ml[prow] = make_float2(live ? ref : -INFINITY, live ? sum : 0.f);
            }
            // drafted elements that were cleared as infinities or NaN
            uint32_t back = 0u;
            if (w.drafted(nc - 1)) {
#pragma unroll
                for (int k = 0; k < 16; ++k) back |= badw[buf * 16 + k];
            }
            if (__any_sync(kFull, in)) {
#pragma unroll 1
                for (int c0 = 0; c0 < G::kHalves * 64; c0 += 16) {
                    const int col = wg * G::kHalves * 64 + c0;            // of O's columns here
                    const int d = (col >> 7) * 256 + kh * 128 + (col & 127);
                    uint32_t o[16];
                    umma::tmem_ld16(lanes + G::kColO + (uint32_t)col, o);
                    umma::tmem_wait_ld();
                    float v[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = live ? __uint_as_float(o[k]) * z : 0.f;
                    if (back && live) {
                        for (int k4 = 0; k4 < 4; ++k4) {
                            uint32_t b = (badw[buf * 16 + k4] | badw[buf * 16 + 4 + k4] | badw[buf * 16 + 8 + k4] | badw[buf * 16 + 12 + k4]) &
                                         bits_at(seen, 32 * k4);
                            for (; b != 0u; b &= b - 1u) {
                                const int pos = w.q.base + 32 * k4 + __ffs(b) - 1;
                                const int blk = __ldg(p.bt + (size_t)w.s * p.max_blocks + pos / kBlock);
                                if (blk < 0 || blk >= p.num_blocks) continue;
                                const uint16_t* src = p.cache + ((size_t)blk * kBlock + pos % kBlock) * (LAT + p.R) + d;
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    if ((__ldg(src + k) & 0x7f80u) == 0x7f80u) v[k] = __uint_as_float(0x7fffffffu);
                            }
                        }
                    }
                    if (!in) continue;
                    if (whole) {
                        uint16_t* dst = p.out + ((size_t)w.q.t0 * p.H + r) * LAT + d;
#pragma unroll
                        for (int k = 0; k < 16; k += 8)
                            *reinterpret_cast<uint4*>(dst + k) =
                                make_uint4(pack_bf16x2(v[k], v[k + 1]), pack_bf16x2(v[k + 2], v[k + 3]),
                                           pack_bf16x2(v[k + 4], v[k + 5]), pack_bf16x2(v[k + 6], v[k + 7]));
                    } else {
                        // (four elements of a row, then those of the next: lanes are rows)
                        float4* dst = reinterpret_cast<float4*>(p.part_o) + (prow - rank * kRows - row) * (LAT / 4) +
                                      (d / 4) * kTile + rank * kRows + row;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            dst[k * kTile] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                    }
                }
            }
            if (tid == 0 && rank == 0 && w.j == 0 && !whole) {
                // the pair with the first pages says where the partials are
                const int last = (int)(((long long)flat + w.q.nb - 1) / misc[M_Q]);
                p.meta[pair] = make_int4(w.s, w.tile, last - pair + 1, min(rows - w.tile * kTile, kTile));
            }
            flat += w.np + kExtraPages;
            g0 += nc;
            umma::fence_before_sync();
            // (the sums have been read before the next maxima are written: the meetings between)
            __syncwarp();
            if (lane == 0) {
                arrive_remote(lead(G::B_OFREE));
                arrive_remote(map_rank(bar(G::B_EPI + buf), 0u));
                arrive_remote(map_rank(bar(G::B_EPI + buf), 1u));
            }
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    cluster_sync();
    // nothing is under way in either CTA's memory when the pair ends: the copies of a pair that ran
    // to its end were all waited for by the MMA warps, and count on the first CTA's barriers
    if (misc[M_ABORT]) {                 // (give_up: both CTAs')
        if (rank == 0 && warp == G::kKWarp && lane == 0) {
            const volatile int* n = misc + M_ISSUED;
            land<1>(n, 2, [&](int) { return bar(G::B_QFULL); });
            for (int k = 0; k < G::kG1; ++k)
                land<G::kSlots>(n + 2 * (1 + k), 2, [&](int g) { return bar(G::B_KFULL + slot(g) * G::kG1 + k); });
            for (int h = 0; h < 2; ++h)
                land<G::kSlots>(n + 2 * (1 + G::kG1 + h), 2, [&](int g) { return bar(G::B_VREADY + slot(g) * 2 + h); });
        }
        __syncwarp();
        cluster_sync();
    }
    if (warp == G::kMmaWarp) {
        umma::fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G::kTmemCols) : "memory");
    }
}

// ------------------------------------------------------------------------- merge

constexpr int kMaxWorkers = 256;
// Parts of a tile, by workers and tiles, from which the warps share them out.  (4 x 131072 tokens,
// 39 parts: four warps, each all parts of a quarter of the row 139 us, a part each in turn 137,
// eight warps 125; 32 x 8192, 3 to 4 parts: a CTA for four pieces 85, for one 88.)
constexpr int kMergeSplit = 8;

constexpr int merge_warps(bool split) { return split ? 8 : 4; }

// Parts of a tile of few rows, likewise, from which a lane has more parts' loads under way, eight
// instead of two, and a CTA more registers.  (32 x 8192, 16 heads, 5 to 6 parts: 65.7 us with eight, 1
// more with four, 69 with two; 64 x 4096, 64 heads, 2 to 3 parts: 3 more with eight than with two.)
constexpr int kMergeWide = 4;

constexpr int merge_parts(bool wide) { return wide ? 8 : 2; }

// What a row gets that has no weight: NaN if it sees a position (its scores were -inf alone).
__device__ __forceinline__ float weightless(const LatentParams& p, int s, int r)
{
    const SeqInfo q = seq_info(p, s, false);
    uint32_t seen[4];
    if (!seen_nodes(p, q.t0, row_node(p, r), nullptr, seen)) return 0.f;
    bool any = q.base > 0;
    for (int k = 0; k < 4; ++k) any = any || (seen[k] & low_bits(q.L - 32 * k)) != 0u;
    return any ? __uint_as_float(0x7fffffffu) : 0.f;
}

// CTA (e, piece): a piece of the e-th tile that has parts, in the order of the workers that
// wrote its first part.  A warp reads 64 elements of 8 rows, where fours of the rows'
// elements lie together, or a row (BY_ROW), where its elements do, a few parts at a time
// with a running (max, sum).  Few parts: the warps have different elements.  Many (SPLIT): they
// take the parts in turn, and their results are joined in the warps' order.
template <int LAT, bool BY_ROW, bool SPLIT, bool WIDE>
__global__ void __launch_bounds__(merge_warps(SPLIT) * 32, SPLIT ? 4 : WIDE ? 2 : 8) paged_latent_merge_kernel(const LatentParams p)
{
    constexpr int kMergeWarps = merge_warps(SPLIT);
    constexpr int kFours = LAT / 4, kN = BY_ROW ? LAT / 128 : 4;     // fours of a row; of a lane
    constexpr int kRounds = (kMaxWorkers + kMergeWarps * 32 - 1) / (kMergeWarps * 32);
    __shared__ int4 s_meta;
    __shared__ int s_x, s_count[kRounds][kMergeWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = p.tile_rows;
    pdl_wait();
    pdl_launch_dependents();
    int4 mine[kRounds];
    unsigned first[kRounds];                             // workers that wrote the first part of a tile
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
        const int x = q * kMergeWarps * 32 + tid;
        mine[q] = x < p.workers ? p.meta[x] : make_int4(0, 0, 0, 0);
        first[q] = __ballot_sync(kFull, mine[q].z > 1);
        if (lane == 0) s_count[q][warp] = __popc(first[q]);
    }
    if (tid == 0) s_x = -1;
    __syncthreads();
    int n = 0;
#pragma unroll
    for (int q = 0; q < kRounds; ++q)
#pragma unroll
        for (int v = 0; v < kMergeWarps; ++v) {
            if (v == warp && ((first[q] >> lane) & 1u) &&
                n + __popc(first[q] & ((1u << lane) - 1u)) == (int)blockIdx.x) {
                s_meta = mine[q];
                s_x = q * kMergeWarps * 32 + tid;
            }
            n += s_count[q][v];
        }
    __syncthreads();
    const int x = s_x;
    if (x < 0) return;
    const int4 meta = s_meta;
    const int parts = meta.z;
    // this warp's piece; this lane's row, its first four of elements and the next ones' distance
    const int sub = SPLIT ? blockIdx.y : blockIdx.y * kMergeWarps + warp;
    constexpr int kStep = BY_ROW ? 32 : 4;
    const int row = BY_ROW ? sub : sub / (LAT / 64) * 8 + (lane & 7);
    const int four = BY_ROW ? lane : sub % (LAT / 64) * 16 + (lane >> 3);
    const bool any_row = (BY_ROW ? row : row & ~7) < meta.w;
    const int t0 = p.starts ? __ldg(p.starts + meta.x) : meta.x;
    // part i: the first worker's second slot, then the first slots
    auto slot = [&](int i) { return ((size_t)(x + i) * 2 + (i == 0 ? 1 : 0)) * R; };
    float M = -INFINITY, l = 0.f, acc[kN][4];
#pragma unroll
    for (int k = 0; k < kN; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.f;
    constexpr int kStride = SPLIT ? kMergeWarps : 1, kParts = merge_parts(WIDE);
    for (int i = SPLIT ? warp : 0; any_row && i < parts; i += kParts * kStride) {
        float2 ml[kParts];
        float4 o[kParts][kN];
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
            const bool there = i + h * kStride < parts;
            const size_t at = slot(there ? i + h * kStride : i);
            ml[h] = there ? p.part_ml[at + row] : make_float2(-INFINITY, 0.f);
            const float4* src = reinterpret_cast<const float4*>(p.part_o) + at * kFours;
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                const int f = four + kStep * k;
                o[h][k] = there ? src[BY_ROW ? row * kFours + f : f * R + row] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        float top = M, a[kParts];
#pragma unroll
        for (int h = 0; h < kParts; ++h) top = fmaxf(top, ml[h].x);
        // a part that saw nothing weighs nothing (its maximum is -inf)
        const float w = M == -INFINITY ? 0.f : ex2(M - top);
        M = top;
        l *= w;
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
            a[h] = ml[h].x == -INFINITY ? 0.f : ex2(ml[h].x - top);
            l += ml[h].y * a[h];
        }
#pragma unroll
        for (int k = 0; k < kN; ++k) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[k][e] *= w;
#pragma unroll
            for (int h = 0; h < kParts; ++h) {
                acc[k][0] += o[h][k].x * a[h];
                acc[k][1] += o[h][k].y * a[h];
                acc[k][2] += o[h][k].z * a[h];
                acc[k][3] += o[h][k].w * a[h];
            }
        }
    }
    if constexpr (SPLIT) {
        __shared__ float4 s_acc[kMergeWarps][kN][32];
        __shared__ float2 s_ml[kMergeWarps][32];
#pragma unroll
        for (int k = 0; k < kN; ++k) s_acc[warp][k][lane] = make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
        s_ml[warp][lane] = make_float2(M, l);
        __syncthreads();
        M = -INFINITY;
#pragma unroll
        for (int q = 0; q < kMergeWarps; ++q) M = fmaxf(M, s_ml[q][lane].x);
        l = 0.f;
        acc[0][0] = acc[0][1] = acc[0][2] = acc[0][3] = 0.f;
        // (warp k joins the warps' k-th fours)
#pragma unroll
        for (int q = 0; q < kMergeWarps; ++q) {
            const float2 ml = s_ml[q][lane];
            const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            l += ml.y * w;
            if (warp < kN) {
                const float4 o = s_acc[q][warp < kN ? warp : 0][lane];
                acc[0][0] += o.x * w;
                acc[0][1] += o.y * w;
                acc[0][2] += o.z * w;
                acc[0][3] += o.w * w;
            }
        }
    }
    if (row >= meta.w || (SPLIT && warp >= kN)) return;
    const int r = meta.y * R + row;
    const float none = l == 0.f ? weightless(p, meta.x, r) : 0.f, inv = 1.f / l;
    uint2* dst = reinterpret_cast<uint2*>(p.out + ((size_t)t0 * p.H + r) * LAT);
#pragma unroll
    for (int k = 0; k < (SPLIT ? 1 : kN); ++k) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = l == 0.f ? none : acc[k][e] * inv;
        dst[four + kStep * (SPLIT ? warp : k)] = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
}

// -------------------------------------------------------------------------- host

int check_latent_shape(int num_seqs, int max_nodes, int H, int L, int R)
{
    if (num_seqs < 0 || max_nodes < 1 || H <= 0 || L <= 0 || R <= 0) return KV_ERR_INVALID_ARG;
    if (max_nodes > KV_TREE_MAX_NODES) return KV_ERR_TOO_LARGE;
    if (H > 128 || (L != 256 && L != 512) || (R != 32 && R != 64)) return KV_ERR_UNSUPPORTED;
    return KV_OK;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// The kernel that serves a shape, by its rows, and the workspace: partial outputs, their
// (max, sum) and the table of them.
struct LatentPlan {
    bool few;
    int workers, rows;          // CTAs or pairs of them, rows of their tiles
    size_t o, ml, meta, total;
};

LatentPlan latent_plan(int max_nodes, int H, int L)
{
    LatentPlan t;
    const int sms = num_sms_current();
    t.few = max_nodes * H <= kLatentFew;
    t.rows = t.few ? kLatentFew : kTile;
    t.workers = std::min(kMaxWorkers, t.few ? sms : std::max(1, sms / 2));
    // (the rows of all workers' tiles are as many by either, so that a workspace for more
    // nodes serves fewer)
    const size_t slots = (size_t)std::max(2, sms) * 2 * kLatentFew;
    t.o = 0;
    t.ml = t.o + up256(slots * L * sizeof(float));
    t.meta = t.ml + up256(slots * sizeof(float2));
    t.total = t.meta + up256((size_t)sms * sizeof(int4));
    return t;
}

std::mutex g_latent_mu;

template <int LAT>
int launch_many(const LatentParams& p, const void* q, const void* cache, cudaStream_t st)
{
    using G = Geo<LAT>;
    const int W = LAT + p.R;
    const long long qrows = (long long)p.total * p.H, krows = (long long)p.num_blocks * kBlock;
    CUtensorMap mq, mqr, mk, mkr, mv;
    if (int rc = latent_column_map(&mq, q, qrows, W, G::kCols, kRows, 4)) return rc;
    if (int rc = latent_row_map(&mqr, q, qrows, W, kRows)) return rc;
    if (int rc = latent_column_map(&mk, cache, krows, W, G::kCols, 8, 4)) return rc;
    if (int rc = latent_row_map(&mkr, cache, krows, W, kBlock)) return rc;
    if (int rc = latent_column_map(&mv, cache, krows, W, G::kCols, kBlock, 2)) return rc;
    static bool ready[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KV_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_latent_mu);
        if (!ready[dev]) {
            if (cudaFuncSetAttribute(paged_latent_kernel<LAT>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem) !=
                cudaSuccess)
                return KV_ERR_CUDA;
            ready[dev] = true;
        }
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * p.workers));
    cfg.blockDim = dim3(G::kThreads);
    cfg.dynamicSmemBytes = G::kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_latent_kernel<LAT>, mq, mqr, mk, mkr, mv, p) == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

template <int LAT, bool BY_ROW, bool SPLIT, bool WIDE = false>
int launch_merge(const LatentParams& p, int tiles, int rows, cudaStream_t st)
{
    constexpr int kMergeWarps = merge_warps(SPLIT);
    const int pieces = BY_ROW ? rows : (rows + 7) / 8 * (LAT / 64);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles, (unsigned)(SPLIT ? pieces : (pieces + kMergeWarps - 1) / kMergeWarps));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_latent_merge_kernel<LAT, BY_ROW, SPLIT, WIDE>, p) == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

template <int LAT>
int launch_all(const LatentParams& p, bool few, const void* q, const void* cache, cudaStream_t st)
{
    if (few) {
        if (latent_small_launch(p, q, cache, LAT, st) != cudaSuccess) return KV_ERR_CUDA;
    } else if (int rc = launch_many<LAT>(p, q, cache, st)) {
        return rc;
    }
    // the tiles that may have parts: no more than there are, nor than workers
    const long long all = (long long)p.B * ((p.max_nodes * p.H + p.tile_rows - 1) / p.tile_rows);
    const int tiles = (int)std::min<long long>(all, p.workers), rows = std::min(p.max_nodes * p.H, p.tile_rows);
    const bool split = p.workers / tiles >= kMergeSplit;
    if (few && !split && p.workers / tiles >= kMergeWide) return launch_merge<LAT, true, false, true>(p, tiles, rows, st);
    if (few)
        return split ? launch_merge<LAT, true, true>(p, tiles, rows, st) : launch_merge<LAT, true, false>(p, tiles, rows, st);
    return split ? launch_merge<LAT, false, true>(p, tiles, rows, st) : launch_merge<LAT, false, false>(p, tiles, rows, st);
}

}  // namespace

// Rows of W elements, as boxes of box_rows rows x box_cols 64-element columns with the
// 128-byte swizzle: column by column in shared memory.
int latent_column_map(CUtensorMap* map, const void* base, long long rows, int W, int cols, int box_rows, int box_cols)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    if (int rc = map_encoder(enc)) return rc;
    cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)cols};
    cuuint64_t strides[2] = {(cuuint64_t)W * 2, 128};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_cols};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? KV_OK
               : KV_ERR_CUDA;
}

// The same rows as they are, in boxes of 64 elements: of the one that starts at W - R, what
// lies behind the row is zeros.
int latent_row_map(CUtensorMap* map, const void* base, long long rows, int W, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    if (int rc = map_encoder(enc)) return rc;
    cuuint64_t dims[2] = {(cuuint64_t)W, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)W * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? KV_OK
               : KV_ERR_CUDA;
}

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
    *bytes = latent_plan(max_nodes, num_q_heads, latent_dim).total;
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
    // flat work indices, tensor-map rows and positions must fit in int32
    const long long tiles = ((long long)max_nodes * num_q_heads + kTile - 1) / kTile;
    if ((long long)total_nodes * num_q_heads >= INT_MAX - 256 || (long long)num_blocks * kBlock >= INT_MAX - 256 ||
        (long long)max_blocks_per_seq * kBlock >= INT_MAX ||
        ((long long)max_blocks_per_seq + 2 * kExtraPages) * num_seqs >= INT_MAX / tiles)
        return KV_ERR_UNSUPPORTED;
    const LatentPlan t = latent_plan(max_nodes, num_q_heads, latent_dim);
    if (workspace_bytes < t.total) return KV_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    LatentParams p;
    p.out = static_cast<uint16_t*>(out);
    p.cache = static_cast<const uint16_t*>(cache);
    p.bt = block_tables;
    p.ctx = context_lens;
    p.starts = node_starts;
    p.parents = node_starts ? parents : nullptr;
    p.B = num_seqs;
    p.total = total_nodes;
    p.max_nodes = max_nodes;
    p.H = num_q_heads;
    p.R = rope_dim;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.h_magic = num_q_heads == 1 ? 0u : 0xffffffffu / (uint32_t)num_q_heads + 1u;
    p.sl2 = scale * 1.4426950408889634f;
    p.test_stall = test_stall_cycles();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    g_launched.note();
    p.part_o = reinterpret_cast<float*>(ws + t.o);
    p.part_ml = reinterpret_cast<float2*>(ws + t.ml);
    p.meta = reinterpret_cast<int4*>(ws + t.meta);
    p.workers = t.workers;
    p.tile_rows = t.rows;
    return latent_dim == 512 ? launch_all<512>(p, t.few, q, cache, st) : launch_all<256>(p, t.few, q, cache, st);
}
