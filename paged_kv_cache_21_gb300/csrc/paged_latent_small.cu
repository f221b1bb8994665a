// paged_latent_attention for calls of at most 64 query rows (tokens times heads) a sequence.
//
// The mathematics is paged_latent.cu's.  One CTA an SM goes over pages in groups of 64
// tokens (4 pages).  A page's rows are copied to shared memory once and read there as K and
// as V:
//     S = Q K^T       (64 rows x 64 tokens, K as it lies there),
//     O^T += V^T P^T  (L x 64 rows, 128 of L a product: V^T as it lies there, P through
//                     shared memory).
//
// What bounds it (L = 512, R = 64): a group's 74 KB take HBM 1.68 us to one SM (6.7 TB/s, 152
// SMs), ~3300 clocks; its products, 36 of M 64, N 64 (45 clocks each at least, measured, 50
// to 58 beside the others) and 16 of M 128, N 64 (49), ~2400 at least.  In the loop a group
// takes ~3650: 90 % of HBM's rate.  32 x 8192 tokens, 16 heads: 66 us (HBM 45; ~6 until the
// first keys are there, ~5 for the ends and the merge); 4 x 131072, 64 rows: 125 (91); one
// context of 128 tokens: 11.9, a chain of short steps.  paged_latent.cu's kernel, which copies
// every byte twice, takes 72, 127 and 12.4 us for them.
//
// How (the rest as in paged_latent.cu):
//  * Shared memory holds Q (74 KB), a ring of two groups (four at L = 256) and P (8 KB).
//    Tokens go by eights of L / 64 + 1 columns of 1 KB (the swizzle's atoms), so that a
//    group's rows are at one stride for the scores, and each page, at the same stride, is
//    one step of the products.  A page is copied anew as soon as its products are done, by a
//    warp of its own; with two groups only, the time from there to the next scores counts,
//    so pages are prefetched to L2 shortly before (32 x 8192, 16 heads: 65.3 us one group ahead,
//    67.2 two, 69.3 three, 71.1 without).
//  * An accumulator of M = 64 has row r in lane 32 (r / 16) + r % 16: each warp weighs 16
//    rows, two threads a row with 32 tokens each.
//  * What must not be multiplied in V is cleared where it lies after the group's scores are
//    computed and before its weights are handed on, by the warps that weigh.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "internal.h"
#include "latent_kernel.cuh"

namespace pkv {

namespace {

constexpr int kPages = 4;                       // pages of a group
constexpr int kRows = kLatentFew;
constexpr int kAheadGroups = 1;                 // groups that are brought to L2 ahead of their copies (above)
// Least range of a CTA.  (With 4, 8, 16: 8 x 4096 at L = 256 16.9, 16.7, 16.4 us; one context of 128
// tokens 10.9, 12.0, 11.9; 32 x 8192 65.4 with each.)
constexpr int kMinPages = 8;
// What a sequence costs beside its pages.  (32 x 8192 tokens, 16 heads: 65.5 us with 6, 65.3 with 12,
// 66.9 with 20; 8 x 4096 at L = 256: 17.7, 16.7, 16.5.)
constexpr int kExtraPages = 12;

template <int LAT>
struct SmallGeo {
    static constexpr int kCols = LAT / 64, kCols1 = kCols + 1;   // 64-element columns; the rotary one
    static constexpr int kTiles = LAT / 128;             // products of M 128 for a page
    static constexpr int kSlots = LAT == 512 ? 2 : 4;    // groups in shared memory
    static constexpr int kWeighWarps = 8, kCopyWarp = 8, kMmaWarp = 12, kAheadWarp = 14;
    static constexpr int kThreads = 16 * 32;             // (one warp is idle: registers go by four)
    static constexpr int kEight = kCols1 * 1024;         // eight tokens: [column][8 tokens][128 B]
    static constexpr int kPage = 2 * kEight;
    static constexpr int kSlot = kPages * kPage;
    static constexpr int kQBytes = kCols1 * kRows * 128; // [column][64 rows][128 B]
    static constexpr int kPBytes = kRows * 128;          // [64 rows][64 tokens]
    static constexpr int kRingOff = 0;
    static constexpr int kQOff = kRingOff + kSlots * kSlot;
    static constexpr int kPOff = kQOff + kQBytes;
    static constexpr int kBarOff = kPOff + kPBytes;
    static constexpr int B_QFULL = 0;                            // Q has landed
    static constexpr int B_QFREE = B_QFULL + 1;                  // the segment's last scores are computed
    static constexpr int B_FULL = B_QFREE + 1;                   // + slot: a group has landed
    static constexpr int B_FREE = B_FULL + kSlots;               // + slot * 4 + page: its products are done
    static constexpr int B_SFULL = B_FREE + kSlots * kPages;     // + buffer: scores
    static constexpr int B_SFREE = B_SFULL + 2;                  // + buffer: they have been read
    static constexpr int B_PFULL = B_SFREE + 2;                  // weights
    static constexpr int B_PFREE = B_PFULL + 1;                  // their products are done
    static constexpr int B_OFREE = B_PFREE + 1;                  // the accumulators have been read
    static constexpr int B_END = B_OFREE + 1;                    // + MMA warp
    static constexpr int B_STALL = B_END + 2;                    // nothing arrives (the test hook)
    static constexpr int kNumBars = B_STALL + 1;
    static constexpr int kMiscOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kBadOff = kMiscOff + (M_WORDS * 4 + 15) / 16 * 16;      // [4] words
    static constexpr int kRedOff = kBadOff + 16;                 // [2][64] floats: maxima, sums
    static constexpr int kFacOff = kRedOff + 2 * kRows * 4;      // [64] floats: a row's factor
    static constexpr int kEnd = kFacOff + kRows * 4;
    static constexpr int kSmem = kEnd;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static_assert(kPages + 1 <= kCopiers, "misc words");
    // tensor memory: two buffers of S, then O^T
    static constexpr uint32_t kColO = 128, kTmemCols = kColO + kTiles * kRows <= 256 ? 256 : 512;
};

// Bounded wait that also gives up when another role of the CTA has given up.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* misc)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (misc[M_ABORT]) return false;
        if (clock64() - t0 > kWaitLimit) {
            misc[M_ABORT] = 1;
            raise_flag(&g_latent_err, KV_DEVERR_PIPELINE_TIMEOUT, blockIdx.x);
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* misc)
{
    return __all_sync(kFull, wait_bar(bar, parity, misc));
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

template <int LAT>
__global__ void __launch_bounds__(SmallGeo<LAT>::kThreads, 1)
paged_latent_small_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qr,
                          const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_kr,
                          const LatentParams p)
{
    using G = SmallGeo<LAT>;
    extern __shared__ __align__(1024) uint8_t gb[];
    const uint32_t sb = smem_u32(gb);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    volatile int* misc = reinterpret_cast<volatile int*>(gb + G::kMiscOff);
    // (the swizzle wants the base that the launch gives where there is no static shared memory)
    if (sb & 1023u) {
        if (tid == 0) raise_flag(&g_latent_err, KV_DEVERR_PIPELINE_TIMEOUT, sb);
        return;
    }
    auto bar = [&](int i) -> uint32_t { return sb + (uint32_t)(G::kBarOff + 8 * i); };
    // group g: its slot and the parity of its pass
    auto slot = [](int g) -> int { return (int)((uint32_t)g % G::kSlots); };
    auto pass = [](int g) -> uint32_t { return (uint32_t)g / G::kSlots & 1u; };

    if (tid == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_kr);
        mbar_init(bar(G::B_QFULL), 1);
        mbar_init(bar(G::B_QFREE), 1);
        for (int i = 0; i < G::kSlots; ++i) mbar_init(bar(G::B_FULL + i), kPages);
        for (int i = 0; i < G::kSlots * kPages; ++i) mbar_init(bar(G::B_FREE + i), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(G::B_SFULL + i), 1);
            mbar_init(bar(G::B_SFREE + i), G::kWeighWarps);
            mbar_init(bar(G::B_END + i), 1);
        }
        mbar_init(bar(G::B_PFULL), G::kWeighWarps);
        mbar_init(bar(G::B_PFREE), 1);
        mbar_init(bar(G::B_OFREE), G::kWeighWarps);
        mbar_init(bar(G::B_STALL), 1);
        misc[M_ABORT] = 0;
        misc[M_SEEN] = 0;
        fence_mbar_init();
    }
    // (all this while the kernel before drains)
    if (warp == G::kMmaWarp) {
        umma::tmem_alloc(sb + G::kMiscOff + 4 * M_TMEM, G::kTmemCols);
        umma::tmem_relinquish();
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    pdl_launch_dependents();
    pdl_wait();
    cut_work<G::kThreads>(p, misc, kMinPages, kExtraPages, cta, cta == 0, tid);
    const uint32_t tmem = (uint32_t)misc[M_TMEM];

    if (warp >= G::kCopyWarp && warp < G::kCopyWarp + kPages) {
        // --------------------- Q, and the pages: a warp for each of a group's
        const int page = warp - G::kCopyWarp;
        int g = 0, queries = 0;
        bool ok = true;
        for (Walk<kPages> w(p, misc); ok && w.more(); w.next(p)) {
            if (page == 0) {
                if (w.seg > 0) ok = wait_warp(bar(G::B_QFREE), (uint32_t)((w.seg - 1) & 1), misc);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(G::B_QFULL), (uint32_t)G::kQBytes);
                    const int row = w.q.t0 * p.H;
#pragma unroll
                    for (int k = 0; k < G::kCols; k += 4)
                        tma_load_3d(sb + (uint32_t)(G::kQOff + k * kRows * 128), &tm_q, 0, row, k, bar(G::B_QFULL));
                    tma_load_2d(sb + (uint32_t)(G::kQOff + G::kCols * kRows * 128), &tm_qr, LAT, row, bar(G::B_QFULL));
                }
                ++queries;
                __syncwarp();
            }
            const int32_t* row = p.bt + (size_t)w.s * p.max_blocks + w.j;
            const int nc = w.chunks();
            int ids = lane < w.np ? __ldg(row + lane) : -1;           // pages 0..31 of the segment
            int ahead = 32 + lane < w.np ? __ldg(row + 32 + lane) : -1;
            for (int c = 0; ok && c < nc; ++c, ++g) {
                if (c > 0 && (c & 7) == 0) {
                    ids = ahead;
                    const int at = (c + 8) * kPages + lane;
                    ahead = at < w.np ? __ldg(row + at) : -1;
                }
                const int sl = slot(g);
                const int id = __shfl_sync(kFull, ids, (c & 7) * kPages + page);
                const bool in = page < w.chunk_pages(c), valid = in && id >= 0 && id < p.num_blocks;
                if (g >= G::kSlots && !wait_warp(bar(G::B_FREE + sl * kPages + page), pass(g) ^ 1u, misc)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    if (in && !valid) raise_flag(&g_latent_err, KV_DEVERR_BLOCK_OUT_OF_RANGE, id);
                    if (valid) mbar_arrive_expect_tx(bar(G::B_FULL + sl), (uint32_t)G::kPage);
                    else mbar_arrive(bar(G::B_FULL + sl));
                }
                __syncwarp();
                if (valid && lane < 4) {
                    // the page's two eights: latent columns, rotary column
                    const uint32_t dst = sb + (uint32_t)(G::kRingOff + sl * G::kSlot + page * G::kPage + (lane & 1) * G::kEight);
                    const int y = id * kBlock + 8 * (lane & 1);
                    if (lane < 2) tma_load_3d(dst, &tm_k, 0, y, 0, bar(G::B_FULL + sl));
                    else tma_load_2d(dst + (uint32_t)(G::kCols * 1024), &tm_kr, LAT, y, bar(G::B_FULL + sl));
                }
            }
        }
        if (lane == 0) {
            misc[M_ISSUED + page] = g;
            if (page == 0) misc[M_ISSUED + kPages] = queries;
        }
        __syncwarp();
    } else if (warp == G::kMmaWarp) {
        // ---------------------------------------------------------------- scores
        if (lane == 0) {
            const uint64_t qdesc = umma::smem_desc_sw128(sb + G::kQOff, 16, 1024);
            const uint64_t kdesc = umma::smem_desc_sw128(sb + G::kRingOff, 16, G::kEight);
            constexpr uint32_t idesc = umma::idesc_bf16_f32(64, 64, false, false);
            bool ok = true;
            if (p.test_stall > 0 && range_pages(misc) > 0 && !mbar_wait_bounded(bar(G::B_STALL), 0u, p.test_stall)) {
                misc[M_ABORT] = 1;
                raise_flag(&g_latent_err, KV_DEVERR_PIPELINE_TIMEOUT, blockIdx.x);
                ok = false;
            }
            int g = 0;
            for (Walk<kPages> w(p, misc); ok && w.more(); w.next(p)) {
                const int nc = w.chunks();
                ok = wait_bar(bar(G::B_QFULL), (uint32_t)(w.seg & 1), misc);
                for (int c = 0; ok && c < nc; ++c, ++g) {
                    // the buffer was read for group g - 2
                    if (g >= 2) ok = wait_bar(bar(G::B_SFREE + (g & 1)), (uint32_t)((g >> 1) - 1) & 1u, misc);
                    ok = ok && wait_bar(bar(G::B_FULL + slot(g)), pass(g), misc);
                    if (!ok) break;
                    umma::fence_after_sync();
                    const uint32_t d = tmem + (uint32_t)(64 * (g & 1));
                    const uint64_t kd = kdesc + (uint64_t)((slot(g) * G::kSlot) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4 * G::kCols1; ++kk)
                        umma::mma_bf16_ss(d, qdesc + (uint64_t)(((kk >> 2) * kRows * 128 + (kk & 3) * 32) >> 4),
                                          kd + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), idesc, kk > 0);
                    umma::commit(bar(G::B_SFULL + (g & 1)));
                    if (c + 1 == nc) umma::commit(bar(G::B_QFREE));
                }
            }
            // every MMA issued by this thread is complete before the CTA ends
            umma::commit(bar(G::B_END));
            mbar_wait_bounded(bar(G::B_END), 0u, kWaitLimit);
        }
        __syncwarp();
    } else if (warp == G::kMmaWarp + 1) {
        // -------------------------------------------------------------- products
        if (lane == 0) {
            const uint64_t vdesc = umma::smem_desc_sw128(sb + G::kRingOff, 1024, G::kEight);
            const uint64_t pdesc = umma::smem_desc_sw128(sb + G::kPOff, 16, 1024);
            constexpr uint32_t idesc = umma::idesc_bf16_f32(128, kRows, true, false);
            bool ok = true;
            int g = 0;
            for (Walk<kPages> w(p, misc); ok && w.more(); w.next(p)) {
                const int nc = w.chunks();
                // the accumulators of the segment before have been read
                if (w.seg > 0) ok = wait_bar(bar(G::B_OFREE), (uint32_t)((w.seg - 1) & 1), misc);
                for (int c = 0; ok && c < nc; ++c, ++g) {
                    const int sl = slot(g), np = w.chunk_pages(c);
                    ok = wait_bar(bar(G::B_PFULL), (uint32_t)(g & 1), misc);
                    if (!ok) break;
                    umma::fence_after_sync();
#pragma unroll
                    for (int k = 0; k < kPages; ++k) {
                        if (k < np) {
#pragma unroll
                            for (int t = 0; t < G::kTiles; ++t)
                                umma::mma_bf16_ss(tmem + G::kColO + (uint32_t)(kRows * t),
                                                  vdesc + (uint64_t)((sl * G::kSlot + k * G::kPage + t * 2048) >> 4),
                                                  pdesc + (uint64_t)((k * 32) >> 4), idesc, c + k > 0);
                        }
                        umma::commit(bar(G::B_FREE + sl * kPages + k));
                    }
                    umma::commit(bar(G::B_PFREE));
                }
            }
            umma::commit(bar(G::B_END + 1));
            mbar_wait_bounded(bar(G::B_END + 1), 0u, kWaitLimit);
        }
        __syncwarp();
    } else if (warp == G::kAheadWarp) {
        // ------------------ pages of the groups to come, to L2, a few groups ahead of the copies
        int g = 0;
        bool ok = true;
        for (Walk<kPages> w(p, misc); ok && w.more(); w.next(p)) {
            const int32_t* row = p.bt + (size_t)w.s * p.max_blocks + w.j;
            const int nc = w.chunks();
            // (the first chunks are copied at once)
            for (int a = G::kSlots; ok && a < nc; ++a) {
                if (a > kAheadGroups) ok = __all_sync(kFull, wait_seen(g + a - kAheadGroups - 1, misc));
                const int page = a * kPages + (lane & 3);
                if (ok) prefetch_page(p, page < w.np ? __ldg(row + page) : -1, LAT + p.R, lane >> 2);
            }
            g += nc;
        }
    } else if (warp < G::kWeighWarps) {
        // --------------------------------------------------- weights and output
        const int wq = warp & 3, wg = warp >> 2;
        const int row = wq * 16 + (lane & 15);   // lanes 16..31 have none
        const bool mine = lane < 16;
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        float* red = reinterpret_cast<float*>(gb + G::kRedOff);
        float* fac = reinterpret_cast<float*>(gb + G::kFacOff);
        uint32_t* badw = reinterpret_cast<uint32_t*>(gb + G::kBadOff);
        // sequences without a context: zeros for their nodes
        for (int s = cta; s < p.B; s += gridDim.x) {
            const SeqInfo q = seq_info(p, s, false);
            if (q.L == 0 && q.n > 0) zero_nodes<LAT>(p, q, tid, G::kWeighWarps * 32);
        }
        if (tid == 0) p.meta[cta] = make_int4(0, 0, 0, 0);
        int g0 = 0, flat = misc[M_B0];
        bool ok = true;
        // The eight warps meet: is `x` true anywhere?  Every warp comes to every meeting, also
        // one whose waits have run out, which the others learn there.
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
        // the products of group g are done
        auto used = [&](int g) -> bool { return g < 0 || wait_bar(bar(G::B_PFREE), (uint32_t)(g & 1), misc); };
        for (Walk<kPages> w(p, misc); ok && w.more(); w.next(p)) {
            const int nc = w.chunks(), rows = w.q.n * p.H;
            uint32_t seen[4];
            bool live = mine && row < rows;
            {
                const int i = live ? row_node(p, row) : 0;
                live = seen_nodes(p, w.q.t0, i, w.j == 0 && live ? &g_latent_err : nullptr, seen) && live;
            }
            const bool warp_live = __any_sync(kFull, live);
            float ref = -INFINITY, nref = live ? 0.f : -INFINITY, l[4] = {0.f, 0.f, 0.f, 0.f};
            bool pending = true;                 // a row has no reference yet
            for (int c = 0; c < nc; ++c) {
                const int g = g0 + c;
                ok = __all_sync(kFull, ok && wait_bar(bar(G::B_SFULL + (g & 1)), (uint32_t)((g >> 1) & 1), misc));
                if (tid == 0) misc[M_SEEN] = g + 1;
                umma::fence_after_sync();
                float t[32];
                const int np = w.chunk_pages(c), k0 = wg * 32;           // this thread's first token
                const int p0 = (w.j + c * kPages) * kBlock;              // the group's
                const bool masked = w.drafted(c) || np < kPages;
                if (warp_live) {
                    umma::tmem_ld32(lanes + (uint32_t)(64 * (g & 1) + 32 * wg), *reinterpret_cast<uint32_t(*)[32]>(&t[0]));
                    umma::tmem_wait_ld();
                }
                umma::fence_before_sync();
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(bar(G::B_SFREE + (g & 1)));
                float most = -INFINITY;
                if (warp_live) {
                    // (the product rounded before the sum: the reference is such a product, and a
                    // fused remainder would grow with it)
                    const u64 f = pack2(p.sl2, p.sl2);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) unpack2(mul2(pack2(t[k], t[k + 1]), f), t[k], t[k + 1]);
                    if (masked) {
                        const int pos = p0 + k0;
                        const uint32_t vis = (low_bits(w.q.base - pos) | bits_at(seen, pos - w.q.base)) &
                                             low_bits(min(w.q.L - pos, np * kBlock - k0));
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
                    if (c == 0 && tid < 4) badw[tid] = 0u;       // (last read before that meeting)
                    if (meet(!ok)) {
                        ok = false;
                        break;
                    }
                    // ---- new references: the largest score of each row in the group
                    float top = -INFINITY;
                    if (warp_live) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) top = max_nan(top, t[k]);
                    }
                    if (mine) red[wg * kRows + row] = top;
                    meet(false);
                    top = max_nan(red[row], red[kRows + row]);
                    // a row whose first scores hold NaN is NaN whatever its reference: 0
                    if (ref == -INFINITY && top != top) top = 0.f;
                    float a = 1.f;
                    if (live && (ref == -INFINITY ? top > -INFINITY : top > ref + kMaxLag)) {
                        a = ref == -INFINITY ? 0.f : ex2(ref - top);
                        ref = top;
                        nref = -top;
                    }
                    if (mine && wg == 0) fac[row] = a;
                    // what has been accumulated follows, once the products under way are done
                    const bool moved = meet(a != 1.f) && c > 0;
                    if (moved) ok = __all_sync(kFull, used(g - 1));
                    pending = meet(live && ref == -INFINITY);
                    if (meet(!ok)) {
                        ok = false;
                        break;
                    }
                    if (moved) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) l[k] *= a;
                        umma::fence_after_sync();
                        // a row is a column of O^T: its factor for all lanes
#pragma unroll 1
                        for (int c0 = 0; c0 < G::kTiles * kRows / 2; c0 += 16) {
                            const int col = wg * (G::kTiles * kRows / 2) + c0;
                            const uint32_t at = lanes + G::kColO + (uint32_t)col;
                            uint32_t o[16];
                            umma::tmem_ld16(at, o);
                            umma::tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * fac[(col & (kRows - 1)) + k]);
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
                // ---- what must not be multiplied: rows behind the context, infinities and NaN
                // of drafted rows (the scores are computed, nothing else reads them as K)
                if (w.drafted(c) && ok) {
                    const int lo = max(0, w.q.base - p0), hi_row = np * kBlock;
                    for (int r = lo + warp; r < hi_row; r += G::kWeighWarps) {
                        const bool tail = p0 + r >= w.q.L;
                        uint32_t found = 0u;
                        for (int x = lane; x < G::kCols * 8; x += 32) {
                            const uint32_t at = sb + (uint32_t)(G::kRingOff + slot(g) * G::kSlot + (r >> 3) * G::kEight +
                                                                (x >> 3) * 1024 + (r & 7) * 128 + (((x & 7) ^ (r & 7)) * 16));
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
                            found |= any;
                        }
                        const int a = p0 + r - w.q.base;
                        if (__any_sync(kFull, found != 0u) && lane == 0) atomicOr(&badw[a >> 5], 1u << (a & 31));
                    }
                }
                // the buffer of P: the products of the group before are done.  (A wait that runs
                // out is told at the next meeting; nothing is written then.)
                ok = __all_sync(kFull, ok && used(g - 1));
                if (ok && warp_live && mine) {
                    const uint32_t pb = sb + (uint32_t)(G::kPOff + row * 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sts128(pb + (uint32_t)(((wg * 4 + k) ^ (row & 7)) * 16),
                               make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]));
                }
                fence_proxy_async_smem();
                umma::fence_before_sync();
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(bar(G::B_PFULL));
            }
            // the warps go on together, or not at all
            if (meet(!ok)) ok = false;
            if (!ok) break;
            // ---- the segment's result
            ok = __all_sync(kFull, used(g0 + nc - 1));
            umma::fence_after_sync();
            if (mine) red[wg * kRows + row] = (l[0] + l[1]) + (l[2] + l[3]);
            if (meet(!ok)) ok = false;
            if (!ok) break;
            const bool whole = w.whole();
            const size_t prow = ((size_t)cta * 2 + (w.j == 0 ? 1 : 0)) * kRows;
            uint32_t back = 0u;                  // drafted rows where something was cleared
            if (w.drafted(nc - 1)) back = badw[0] | badw[1] | badw[2] | badw[3];
            // (those that a row sees: where P was)
            uint32_t* rowbad = reinterpret_cast<uint32_t*>(gb + G::kPOff);
            if (mine && wg == 0) {
                const float sum = red[row] + red[kRows + row];
                float z = 1.f;
                if (whole) {
                    bool any = w.q.base > 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) any = any || (seen[k] & low_bits(w.q.L - 32 * k)) != 0u;
                    // (a row that sees something and weighs nothing had scores of -inf alone)
                    z = live && sum != 0.f ? 1.f / sum : live && any ? __uint_as_float(0x7fffffffu) : 0.f;
                } else if (row < rows) {
                    p.part_ml[prow + row] = make_float2(live ? ref : -INFINITY, live ? sum : 0.f);
                }
                // (a row that is not live may hold anything: told apart by a negative factor)
                fac[row] = live ? z : -1.f;
                if (back) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) rowbad[row * 4 + k] = live ? badw[k] & seen[k] : 0u;
                }
            }
            meet(false);
            // a thread per column of L: 128 a tile
            const int shown = min(rows, kRows);
#pragma unroll 1
            for (int t = wg; t < G::kTiles; t += 2) {
                const int d = t * 128 + wq * 32 + lane;
#pragma unroll 1
                for (int r0 = 0; r0 < shown; r0 += 16) {
                    uint32_t o[16];
                    umma::tmem_ld16(lanes + G::kColO + (uint32_t)(t * kRows + r0), o);
                    float v[16];
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 z = *reinterpret_cast<const float4*>(fac + r0 + k);
                        v[k] = z.x; v[k + 1] = z.y; v[k + 2] = z.z; v[k + 3] = z.w;
                    }
                    umma::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = v[k] < 0.f ? 0.f : __uint_as_float(o[k]) * v[k];
                    if (back) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            if (r0 + k >= shown) continue;
                            for (int k4 = 0; k4 < 4; ++k4) {
                                for (uint32_t b = rowbad[(r0 + k) * 4 + k4]; b != 0u; b &= b - 1u) {
                                    const int pos = w.q.base + 32 * k4 + __ffs(b) - 1;
                                    const int blk = __ldg(p.bt + (size_t)w.s * p.max_blocks + pos / kBlock);
                                    if (blk < 0 || blk >= p.num_blocks) continue;
                                    const uint16_t x = __ldg(p.cache + ((size_t)blk * kBlock + pos % kBlock) * (LAT + p.R) + d);
                                    if ((x & 0x7f80u) == 0x7f80u) v[k] = __uint_as_float(0x7fffffffu);
                                }
                            }
                        }
                    }
                    if (whole) {
                        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.out) + ((size_t)w.q.t0 * p.H + r0) * LAT + d;
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (r0 + k < shown) dst[k * LAT] = __float2bfloat16_rn(v[k]);
                    } else {
                        float* dst = p.part_o + (prow + r0) * LAT + d;
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (r0 + k < shown) dst[k * LAT] = v[k];
                    }
                }
            }
            if (tid == 0 && w.j == 0 && !whole) {
                // the CTA with the first pages says where the partials are
                const int last = (int)(((long long)flat + w.q.nb - 1) / misc[M_Q]);
                p.meta[cta] = make_int4(w.s, 0, last - cta + 1, rows);
            }
            flat += w.np + kExtraPages;
            g0 += nc;
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(G::B_OFREE));
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    // every copy lands before the CTA can end: those of a CTA that ran to its end were all
    // waited for by the MMA warps
    if (misc[M_ABORT] && warp == G::kCopyWarp && lane == 0) {
        land<G::kSlots>(misc + M_ISSUED, kPages, [&](int g) { return bar(G::B_FULL + slot(g)); });
        land<1>(misc + M_ISSUED + kPages, 1, [&](int) { return bar(G::B_QFULL); });
    }
    if (warp == G::kMmaWarp) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, G::kTmemCols);
    }
}

std::mutex g_small_mu;

template <int LAT>
cudaError_t launch(const LatentParams& p, const void* q, const void* cache, cudaStream_t st)
{
    using G = SmallGeo<LAT>;
    const int W = LAT + p.R;
    const long long qrows = (long long)p.total * p.H, krows = (long long)p.num_blocks * kBlock;
    CUtensorMap mq, mqr, mk, mkr;
    if (latent_column_map(&mq, q, qrows, W, G::kCols, kRows, 4) || latent_row_map(&mqr, q, qrows, W, kRows) ||
        latent_column_map(&mk, cache, krows, W, G::kCols, 8, G::kCols) || latent_row_map(&mkr, cache, krows, W, 8))
        return cudaErrorUnknown;
    static bool ready[64] = {};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(g_small_mu);
        if (!ready[dev]) {
            if (cudaError_t e = cudaFuncSetAttribute(paged_latent_small_kernel<LAT>,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem))
                return e;
            ready[dev] = true;
        }
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.workers);
    cfg.blockDim = dim3(G::kThreads);
    cfg.dynamicSmemBytes = G::kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_latent_small_kernel<LAT>, mq, mqr, mk, mkr, p);
}

}  // namespace

cudaError_t latent_small_launch(const LatentParams& p, const void* q, const void* cache, int latent_dim, cudaStream_t st)
{
    g_launched.note();
    return latent_dim == 512 ? launch<512>(p, q, cache, st) : launch<256>(p, q, cache, st);
}

int latent_small_read_error(unsigned* flags, long long* detail) { return g_launched.take_error(g_latent_err, flags, detail); }

}  // namespace pkv
