// paged_tree_attention: attention of trees of drafted tokens over a
// block-paged KV cache, on the 5th-generation tensor cores of sm_103a.
//
// What is computed, for node i of sequence s and query head h (KV head h / G):
//     out[i][h] = softmax_j(scale * q[i][h] . K_j) V_j
// over the positions j that the node sees: the committed tokens, its ancestors
// in the drafted tree and itself (the formula of "KV Cache" (heepie.pages.dev),
// section "Self-Attention"; keys through the block table of "KV Cache, Flash
// Attention and inference optimization", section "PagedAttention"; the running
// (max, sum) softmax of its section "Numerical trick").
//
// What bounds it: with n nodes the K and V of a sequence are read once for all
// n * G query rows of a KV head.  Up to 64 rows the time is that of the bytes; 128 rows
// take 1.5 times that, 256 rows twice, for the chain from scores to products (below).
//
// This file holds the kernel for more than 64 rows, the kernel that joins
// partial results, and the entry points; paged_tree_small.cu the kernel for up
// to 64 rows.  A call whose trees may have either launches both, each for its
// sequences.
//
// How:
//  * The rows of a KV head's nodes (row r = node * G + head) fill tiles of 128
//    rows, one MMA's M.  A CTA works on one tile (TILES == 1) or two (TILES ==
//    2, when a tree may have more than 128 rows); more tiles than that are
//    served by as many teams of CTAs, which cut the same keys the same way, so
//    that the repeated reads of a tile of keys come at about the same time and
//    hit L2.
//  * One persistent CTA per SM takes a contiguous range of the flat (sequence,
//    KV head, page) list (cut_work) and consumes it in chunks of up to 8 pages
//    (128 keys).  A warp each streams K and V into rings with TMA (E4M3: one warp
//    both, and two warps widen V).
//  * Two streams work side by side, each with its half of tensor memory: the
//    scores S (128 columns), overwritten in place by the weights P, and the
//    accumulator O.  With TILES == 2 a stream has its own row tile and both
//    consume every chunk; with TILES == 1 they take the chunks in turn and
//    their two results are joined at the end of the range.
//  * A row has two threads, in two of the stream's eight softmax warps: half of
//    the chunk's keys each, 64 scores that stay in registers from the maximum (the
//    two meet in shared memory) to the weights.
//  * One thread issues all MMAs.  A stream's products are followed by its own next
//    scores at once, so that one stream's softmax runs while the other has the
//    tensor cores: with an MMA thread a stream they ran S S PV PV, and both softmax
//    phases contended for the same units (458 us against 361, at 64 nodes x 4 heads
//    of 32 x 8192 tokens).  A commit costs this thread ~100 clocks and a test of a
//    barrier as much, so slots are released by plain arrivals behind a wait that is
//    due anyway, and what is usually ready is waited for ahead (361 -> 331 us).
//  * S = Q K^T with K as it lies in the ring; O += P V with P from tensor memory.
//    P is f16 for an E4M3 cache (whose V is widened to f16, which holds every code
//    exactly); for a bf16 cache it is bf16, in high and low parts (16 bits, two
//    products) for a float32 output (LOW).  For a bf16 output the high part
//    alone, since the second product costs a fifth (402 us against 328): 2^-8 of each
//    weight at most, of either sign, which over many keys comes to about what the
//    output's own rounding does (the largest error of 32 x 8192 tokens, 64 nodes goes
//    from 0.0017 to 0.0023).  The sum is that of the rounded weights.
//  * Measured at 64 nodes x 4 heads of 32 x 8192 tokens: 328 us; the bytes take 164,
//    the products 149 at the tensor cores' rate, 117 the exponentials.  A 128-key
//    chunk takes ~4900 clocks; a stream's chain is 590 to issue S, 230 until it is
//    seen, ~2400 of softmax (200 until the scores are read, 360 maximum, 200 for
//    the halves to meet, 900 weights; four warps share a scheduler), 650 to issue
//    P V, 450 until its end is seen.  P in tensor memory of its own with S two
//    chunks ahead removes the chain but has both softmax phases contend again (332),
//    and takes two waits a chunk for a float32 output (846 against 397 then); 64-key
//    pieces of S cost as many MMA clocks as 128 (530 against 499 then); products of
//    half the keys while the others are weighed cost what they gain (327).
//  * Only the chunks that reach the drafted positions need masks; there a prep warp
//    (or the widening warps) first zeroes the V rows behind the context and the
//    infinities and NaN of drafted rows, which 0 * V would spread to nodes that
//    do not see them; nodes that do see them get them added back at the end.
//  * A range that holds all pages of a (sequence, KV head) writes the output;
//    else unnormalised partials with their (max, sum) go to the workspace, and
//    a second kernel joins them by the log-sum-exp rule, in CTA order.
//  * Every wait is bounded; a time-out sets KV_DEVERR_PIPELINE_TIMEOUT and ends
//    every role of the CTA, which still waits for its copies and MMAs in flight
//    before it frees tensor memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "cache_map.h"
#include "internal.h"
#include "tree_kernel.cuh"

namespace pkv {

namespace {

constexpr int kTile = 128;                      // rows of a tile: M of every MMA
constexpr uint32_t kTmemCols = 512;             // S0, S1, O0, O1: 128 columns each
constexpr int kSoftWarps = 16;                  // softmax: 2 streams x 2 halves of the keys x 4

template <int D, bool FP8, int TILES>
struct Geo {
    static constexpr int kD = D;
    static constexpr bool kFp8 = FP8;
    static constexpr int kCopyWarp = kSoftWarps;
    static constexpr int kMmaWarp = kCopyWarp + 1;
    static constexpr int kPrepWarp = kMmaWarp + 1;           // first of the prep / widening warps
    static constexpr int kPrepWarps = FP8 ? 2 : 1;
    static constexpr int kCopyV = kPrepWarp + 1;             // (bf16) the copies of V
    static constexpr int kWarps = kPrepWarp + 2;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kBoxes = D / 64;                    // 128-byte column groups of a row
    static constexpr int kSlot = kBoxes * kRegion;           // K or V of a chunk, 2 bytes each
    static constexpr int kQTile = FP8 ? kQueryParts * kTile * D : kBoxes * kTile * 128;
    static constexpr int kWords = kN / 32;                   // words of a node's bits
    static constexpr int kPageBytes = kBlock * D * (FP8 ? 1 : 2);
    static constexpr int kRawSlot = kPages * kBlock * D;     // E4M3 codes of K or V of a chunk
    static constexpr int kScale = 128 / D;
    // the two streams take the chunks in turn, or both take each
    static constexpr int kChunkStep = TILES == 1 ? 2 : 1;
    // (E4M3: two tiles of queries in three parts leave room for less)
    static constexpr int kKSlots = (FP8 && TILES == 1 ? 3 : 2) * kScale;
    static constexpr int kVSlots = (!FP8 && TILES == 1 ? 3 : 2) * kScale;
    static constexpr int kRawV = !FP8 ? 0 : (TILES == 1 ? 2 : 1) * kScale;
    static constexpr int kLoadBytes = FP8 ? kRawSlot : kSlot;
    static constexpr int kQOff = 0;
    static constexpr int kKOff = kQOff + TILES * kQTile;
    static constexpr int kVOff = kKOff + kKSlots * kLoadBytes;
    static constexpr int kRawOff = kVOff + kVSlots * kSlot;
    static constexpr int kBarOff = kRawOff + kRawV * kRawSlot;
    static constexpr int kVLoadOff = FP8 ? kRawOff : kVOff;
    // barriers
    static constexpr int kVL = FP8 ? kRawV : kVSlots;
    static constexpr int B_KFULL = 0;                        // + slot: K has landed
    static constexpr int B_KEMPTY = B_KFULL + kKSlots;       // + slot: it may be refilled
    static constexpr int B_VFULL = B_KEMPTY + kKSlots;       // V, or its codes
    static constexpr int B_VEMPTY = B_VFULL + kVL;
    static constexpr int B_VWIDE = B_VEMPTY + kVL;           // (FP8) + slot: widened
    static constexpr int B_VWFREE = B_VWIDE + (FP8 ? kVSlots : 0);
    static constexpr int B_FIX = B_VWFREE + (FP8 ? kVSlots : 0);     // (bf16) + slot: V rows fixed
    using KRing = Ring<kKSlots, B_KFULL, B_KEMPTY>;
    using VLoad = Ring<kVL, B_VFULL, B_VEMPTY>;              // what TMA fills, and what the MMAs read
    using VRing = Ring<kVSlots, FP8 ? B_VWIDE : B_VFULL, FP8 ? B_VWFREE : B_VEMPTY>;
    static constexpr int B_QFULL = B_FIX + (FP8 ? 0 : kVSlots);  // Q and the tree of a segment
    static constexpr int B_QFREE = B_QFULL + 1;              // its last scores are computed
    static constexpr int B_SFULL = B_QFREE + 1;              // + stream
    static constexpr int B_PFULL = B_SFULL + 2;              // + stream
    static constexpr int B_PVDONE = B_PFULL + 2;             // + stream
    static constexpr int B_OFULL = B_PVDONE + 2;             // both accumulators are complete
    static constexpr int B_OFREE = B_OFULL + 1;              // + segment & 1: they have been read
    static constexpr int B_ML = B_OFREE + 2;                 // the streams' (max, sum) are written
    static constexpr int B_MAX = B_ML + 1;                   // + stream * 4 + warp's rows: both maxima are written
    static constexpr int B_END = B_MAX + 8;                  // all MMAs are done
    static constexpr int B_STALL = B_END + 1;                // nothing arrives (the test hook)
    static constexpr int kNumBars = B_STALL + 1;
    static constexpr int kMiscOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kAncOff = kMiscOff + 64;            // [2][kN][4] words
    static constexpr int kPtrOff = kAncOff + 2 * kN * 16;    // [kN] bytes used by pointer jumping
    static constexpr int kPadOff = kPtrOff + kN * 4;         // [2][4] words
    static constexpr int kBadOff = kPadOff + 32;             // [2][kPrepWarps][4] words
    static constexpr int kMaxOff = kBadOff + 2 * kPrepWarps * 16;    // [2 streams][2 halves][kTile] floats
    static constexpr int kMlOff = kMaxOff + 4 * kTile * 4;   // [2 streams][2 halves][kTile] float2
    static constexpr int kQfacOff = kMlOff + 4 * kTile * 8;
    static constexpr int kEnd = kQfacOff + (FP8 ? 2 * TILES * kTile * 4 : 0);
    static constexpr int kSmem = kEnd + 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
};

template <int D, bool FP8, int TILES, bool LOW>
__global__ void __launch_bounds__(Geo<D, FP8, TILES>::kThreads, 1)
paged_tree_kernel(const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const TreeParams p)
{
    using G = Geo<D, FP8, TILES>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sraw = smem_u32(smem_raw);
    const uint32_t sb = (sraw + 1023u) & ~1023u;
    uint8_t* gb = smem_raw + (sb - sraw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int team = blockIdx.x / p.nctas, cta = blockIdx.x - team * p.nctas;
    const int first_row = team * TILES * kTile;
    volatile int* misc = reinterpret_cast<volatile int*>(gb + G::kMiscOff);
    auto bar = [&](int i) -> uint32_t { return sb + (uint32_t)(G::kBarOff + 8 * i); };
    uint32_t* anc = reinterpret_cast<uint32_t*>(gb + G::kAncOff);
    volatile uint32_t* padw = reinterpret_cast<volatile uint32_t*>(gb + G::kPadOff);
    volatile uint32_t* badw = reinterpret_cast<volatile uint32_t*>(gb + G::kBadOff);

    if (tid == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        for (int i = 0; i < G::kKSlots; ++i) {
            mbar_init(bar(G::B_KFULL + i), 1);
            mbar_init(bar(G::B_KEMPTY + i), 1);
        }
        // (a slot of codes is freed by the widening warps, which also fill)
        for (int i = 0; i < G::kVL; ++i) {
            mbar_init(bar(G::B_VFULL + i), 1);
            mbar_init(bar(G::B_VEMPTY + i), FP8 ? G::kPrepWarps : 1);
        }
        for (int i = 0; i < G::kVSlots; ++i) {
            if (FP8) {
                mbar_init(bar(G::B_VWIDE + i), G::kPrepWarps);
                mbar_init(bar(G::B_VWFREE + i), 1);
            } else {
                mbar_init(bar(G::B_FIX + i), 1);
            }
        }
        mbar_init(bar(G::B_QFULL), G::kPrepWarps);
        mbar_init(bar(G::B_QFREE), 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar(G::B_SFULL + w), 1);
            mbar_init(bar(G::B_PFULL + w), 8);
            mbar_init(bar(G::B_PVDONE + w), 1);
            mbar_init(bar(G::B_OFREE + w), kSoftWarps);
        }
        mbar_init(bar(G::B_OFULL), 1);
        mbar_init(bar(G::B_END), 1);
        mbar_init(bar(G::B_ML), kSoftWarps);
        for (int i = 0; i < 8; ++i) mbar_init(bar(G::B_MAX + i), 2);
        mbar_init(bar(G::B_STALL), 1);
        misc[M_ABORT] = 0;
        misc[M_VISSUED] = 0;
        fence_mbar_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    if (warp == G::kMmaWarp) {
        umma::tmem_alloc(sb + G::kMiscOff + 4 * M_TMEM, kTmemCols);
        umma::tmem_relinquish();
    }
    if (warp == G::kCopyWarp) cut_work(p, misc, first_row, cta, p.tidy && blockIdx.x == 0, lane);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = (uint32_t)misc[M_TMEM];

    if (warp == G::kCopyWarp) {
        copy_role<G, FP8 ? 2 : 0>(p, tm_k, tm_v, sb, misc, first_row, lane);
    } else if (!FP8 && warp == G::kCopyV) {
        copy_role<G, 1>(p, tm_k, tm_v, sb, misc, first_row, lane);
    } else if (warp == G::kMmaWarp) {
        // --------------------------------------------------------------- MMAs
        if (lane == 0) {
            const uint32_t qt = sb + (uint32_t)G::kQOff;
            const uint64_t qdesc = FP8 ? code_desc<D>(qt) : umma::smem_desc_sw128(qt, 16, 1024);
            const uint64_t sdesc = FP8 ? code_desc<D>(sb + G::kKOff) : umma::smem_desc_sw128(sb + G::kKOff, 16, 1024);
            const uint64_t vdesc = umma::smem_desc_sw128(sb + G::kVOff, kRegion, 1024);
            constexpr uint32_t idesc_pv = FP8 ? umma::idesc_f16_f32(kTile, D, false, true)
                                              : umma::idesc_bf16_f32(kTile, D, false, true);
            using KR = typename G::KRing;
            using VR = typename G::VRing;
            uint32_t fix_parity = 0;             // bit slot: parity of its next fix
            uint32_t turn[2] = {0u, 0u};         // of a stream: parity of its next weights
            bool used[2] = {false, false};       // it has had some
            int g0 = 0;                          // first chunk of the segment
            bool ok = true;
            if (p.test_stall > 0 && misc[M_CNT] > 0 &&
                !mbar_wait_bounded(bar(G::B_STALL), 0u, p.test_stall)) {
                misc[M_ABORT] = 1;
                raise_flag(&g_tree_err, KV_DEVERR_PIPELINE_TIMEOUT, blockIdx.x);
                ok = false;
            }
            for (Walk w(p, misc, first_row); ok && w.more(); w.next(p, first_row)) {
                const int nc = w.chunks(), seg = w.seg;
                // With TILES == 2 both streams take every chunk (the first alone, if the
                // second tile has no rows), with TILES == 1 they take the chunks in turn.
                // A stream's products are followed by its next scores at once, so that
                // its softmax runs while the other stream has the tensor cores.
                constexpr int kStep = G::kChunkStep;
                const bool two = TILES == 1 || w.q.n * p.G - first_row > kTile;
                auto keys = [&](int c) -> bool {
                    return c >= nc || wait_bar(bar(KR::full(g0 + c)), KR::parity(g0 + c), misc);
                };
                // S = Q K^T of chunk c
                auto scores = [&](auto stream, int c) -> bool {
                    constexpr int st = decltype(stream)::value;
                    const bool closes = TILES == 1 || st == 1 || !two;   // last to read the chunk
                    const int g = g0 + c;
                    // the stream's products of the weights that S overwrites are done
                    if (used[st] && !wait_bar(bar(G::B_PVDONE + st), turn[st] ^ 1u, misc)) return false;
                    // and with them all that was issued before: slots are released by
                    // plain arrivals, which cost less than a commit
                    if (c >= kStep && closes) mbar_arrive(bar(VR::free(g - kStep)));
                    if (c > kStep && (TILES == 1 || st == 0)) mbar_arrive(bar(KR::free(g - 1)));
                    umma::fence_after_sync();
                    const uint32_t tS = tmem + (uint32_t)(128 * st);
                    const uint64_t qd = qdesc + (uint64_t)((TILES == 2 ? st * G::kQTile : 0) >> 4);
                    const uint64_t kd = sdesc + (uint64_t)((KR::slot(g) * G::kLoadBytes) >> 4);
                    const uint32_t keys16 = (uint32_t)(kBlock * w.chunk_pages(c));
                    const uint32_t idesc = FP8 ? umma::idesc_f8_f32(kTile, keys16, true, false)
                                               : umma::idesc_bf16_f32(kTile, keys16, false, false);
                    if constexpr (FP8) {
#pragma unroll
                        for (int part = 0; part < kQueryParts; ++part)
#pragma unroll
                            for (int kk = 0; kk < D / 32; ++kk)
                                umma::mma_f8_ss(tS, qd + (uint64_t)((part * kTile * D + kk * 32) >> 4),
                                                kd + (uint64_t)((kk * 32) >> 4), idesc, part + kk > 0);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            umma::mma_bf16_ss(tS, qd + (uint64_t)(((kk >> 2) * kTile * 128 + (kk & 3) * 32) >> 4),
                                              kd + (uint64_t)(((kk >> 2) * kRegion + (kk & 3) * 32) >> 4), idesc, kk > 0);
                    }
                    umma::commit(bar(G::B_SFULL + st));
                    // (the first chunks' slots may be needed before any products are waited for)
                    if (closes && (c < kStep || c + 1 == nc)) umma::commit(bar(KR::free(g)));
                    if (closes && c + 1 == nc) umma::commit(bar(G::B_QFREE));
                    return true;
                };
                // O += P V of chunk c
                auto products = [&](auto stream, int c) -> bool {
                    constexpr int st = decltype(stream)::value;
                    const bool closes = TILES == 1 || st == 1 || !two;
                    const int g = g0 + c, vs = VR::slot(g), np = w.chunk_pages(c);
                    // what is usually there comes first, the weights last
                    if (TILES == 1 || st == 0) {
                        if (!keys(c + kStep)) return false;
                        if (!wait_bar(bar(VR::full(g)), VR::parity(g), misc)) return false;
                        if (!FP8 && w.drafted(c)) {
                            if (!wait_bar(bar(G::B_FIX + vs), (fix_parity >> vs) & 1u, misc)) return false;
                            fix_parity ^= 1u << vs;
                        }
                    }
                    if (st == 0 && c == 0 && seg > 0 &&
                        !wait_bar(bar(G::B_OFREE + ((seg - 1) & 1)), (uint32_t)(((seg - 1) >> 1) & 1), misc))
                        return false;
                    if (!wait_bar(bar(G::B_PFULL + st), turn[st], misc)) return false;
                    umma::fence_after_sync();
                    const uint32_t tS = tmem + (uint32_t)(128 * st), tO = tmem + 256u + (uint32_t)(128 * st);
                    const uint64_t vd = vdesc + (uint64_t)((vs * G::kSlot) >> 4);
                    const bool first = c < kStep;
                    auto page = [&](int kk) {
                        // the weights of keys 16 kk .. 16 kk + 15: 8 columns of the
                        // 32 that held the scores of 32 keys; their low parts 16 on
                        const uint32_t a = tS + (uint32_t)(32 * (kk >> 1) + 8 * (kk & 1));
                        const uint64_t b = vd + (uint64_t)((kk * kBlock * 128) >> 4);
                        umma::mma_bf16_ts(tO, a, b, idesc_pv, !(first && kk == 0));
                        if (LOW) umma::mma_bf16_ts(tO, a + 16u, b, idesc_pv, true);
                    };
                    if (np == kPages) {
#pragma unroll
                        for (int kk = 0; kk < kPages; ++kk) page(kk);
                    } else {
#pragma unroll 1
                        for (int kk = 0; kk < np; ++kk) page(kk);
                    }
                    umma::commit(bar(G::B_PVDONE + st));
                    if (closes && c + kStep >= nc) umma::commit(bar(VR::free(g)));
                    turn[st] ^= 1u;
                    used[st] = true;
                    return true;
                };
                constexpr std::integral_constant<int, 0> s0{};
                constexpr std::integral_constant<int, 1> s1{};
                ok = wait_bar(bar(G::B_QFULL), (uint32_t)(seg & 1), misc) && keys(0) && scores(s0, 0);
                if (TILES == 1) {
                    if (ok && nc > 1) ok = keys(1) && scores(s1, 1);
                    for (int c = 0; ok && c < nc; c += 2) {
                        ok = products(s0, c) && (c + 2 >= nc || scores(s0, c + 2));
                        if (ok && c + 1 < nc) ok = products(s1, c + 1) && (c + 3 >= nc || scores(s1, c + 3));
                    }
                } else {
                    if (ok && two) ok = scores(s1, 0);
                    for (int c = 0; ok && c < nc; ++c) {
                        ok = products(s0, c) && (c + 1 >= nc || scores(s0, c + 1));
                        if (ok && two) ok = products(s1, c) && (c + 1 >= nc || scores(s1, c + 1));
                    }
                }
                if (!ok) break;
                umma::commit(bar(G::B_OFULL));
                g0 += nc;
            }
            // every MMA issued by this thread is complete before the CTA ends
            umma::commit(bar(G::B_END));
            mbar_wait_bounded(bar(G::B_END), 0u, kWaitLimit);
        }
        __syncwarp();
    } else if (warp >= G::kPrepWarp) {
        // ------------------------- queries, trees, V rows, and widening (E4M3)
        const int pw = warp - G::kPrepWarp;
        int g0 = 0;
        bool ok = true;
        for (Walk w(p, misc, first_row); ok && w.more(); w.next(p, first_row)) {
            const int seg = w.seg, buf = seg & 1, nc = w.chunks(), n = w.q.n;
            // the segment's entry of the tree tables was last read two segments ago
            if (seg >= 2) ok = wait_warp(bar(G::B_OFREE + buf), (uint32_t)(((seg - 2) >> 1) & 1), misc);
            if (ok && seg >= 1) ok = wait_warp(bar(G::B_QFREE), (uint32_t)((seg - 1) & 1), misc);
            if (!ok) break;
            if (lane < 4) badw[(buf * G::kPrepWarps + pw) * 4 + lane] = 0u;
            // ---- the query rows of the team's tiles
            const int rows = min(n * p.G - first_row, TILES * kTile);
            constexpr int C = D / 8, RI = 32 / C;    // 16-byte chunks of a row, rows of an instruction
            const int c = lane % C;
            for (int rb = pw * RI; rb < rows; rb += G::kPrepWarps * RI) {
                const int r = rb + lane / C, rc = min(r, rows - 1);
                const int node = row_node(p, first_row + rc), g = first_row + rc - node * p.G;
                const uint16_t* src =
                    p.q + ((size_t)(w.q.t0 + node) * p.Hq + (size_t)w.h * p.G + g) * D + 8 * c;
                if (!FP8) {
                    const uint32_t dst = sb + (uint32_t)(G::kQOff + (rc >> 7) * G::kQTile + (c >> 3) * kTile * 128) +
                                         region_off(rc & 127, c & 7);
                    if (r < rows) cp_async16(dst, src);
                } else {
                    float up;
                    uint2 parts[kQueryParts];
                    query_e5m2<D>(__ldg(reinterpret_cast<const uint4*>(src)), parts, up);
                    if (r < rows) {
                        const uint32_t at = sb + (uint32_t)(G::kQOff + (rc >> 7) * G::kQTile) + code_off<D>(rc & 127, c);
#pragma unroll
                        for (int part = 0; part < kQueryParts; ++part) sts64(at + (uint32_t)(part * kTile * D), parts[part]);
                        if (c == 0)
                            reinterpret_cast<volatile float*>(gb + G::kQfacOff)[buf * TILES * kTile + r] = up;
                    }
                }
            }
            if (pw == 0) tree_masks<G>(p, w, gb, lane);
            if (!FP8) cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(G::B_QFULL));
            if constexpr (FP8)
                ok = widen<G>(p, w, sb, gb, misc, g0, pw, lane);
            else
                ok = fix_values<G>(p, w, sb, gb, misc, g0, lane);
            g0 += nc;
        }
        if (!FP8) cp_async_wait_all();
    } else {
        // ------------------------------------------------- softmax and output
        const int st = (warp >> 2) & 1;          // stream
        const int half = warp >> 3;              // half of a chunk's keys, and of the output's columns
        const int r = tid & 127;                 // row of the stream's tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + (uint32_t)(128 * st + 64 * half);
        volatile float* maxima = reinterpret_cast<volatile float*>(gb + G::kMaxOff) + st * 2 * kTile + r;
        const uint32_t max_bar = bar(G::B_MAX + (warp & 7));
        const uint32_t tO0 = tmem + lanes + 256u;
        const float v_scale = p.v_scale;
        if (p.tidy && team == 0) zero_empty(p, D, cta, p.nctas, tid, kSoftWarps * 32);
        if (tid == 0) p.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
        int pc = 0, flat = misc[M_B0];
        uint32_t met = 0;                        // parity of the next exchange of maxima
        bool ok = true;
        for (Walk w(p, misc, first_row); ok && w.more(); w.next(p, first_row)) {
            const int seg = w.seg, buf = seg & 1, nc = w.chunks();
            const int r0 = first_row;
            const int rows = w.q.n * p.G - r0;   // rows of this team and those behind it
            const int rt = r + (TILES == 2 ? st * kTile : 0);
            const bool idle = TILES == 2 && st == 1 && rows <= kTile;
            const bool warp_live = (rt & ~31) < rows;
            const bool in = rt < rows;
            const int node = in ? row_node(p, r0 + rt) : 0;
            const uint32_t* am = anc + (buf * kN + node) * 4;
            float m_ref = -INFINITY, l = 0.f;
            float sl2 = p.sl2;
            bool first = true;
            for (int c = TILES == 1 ? st : 0; c < nc && !idle; c += G::kChunkStep) {
                const int np = w.chunk_pages(c);
                const int p0 = (w.j + c * kPages) * kBlock;
                const bool masked = np < kPages || w.drafted(c);
                ok = wait_warp(bar(G::B_SFULL + st), (uint32_t)(pc & 1), misc);
                if (!ok) break;
                if (warp_live) {
                    umma::fence_after_sync();
                    // (a half without keys has scores of an earlier chunk, and sees none)
                    uint32_t sr[2][32];
                    umma::tmem_ld32(tS, sr[0]);
                    umma::tmem_ld32(tS + 32u, sr[1]);
                    umma::tmem_wait_ld();
                    if (FP8 && first)
                        sl2 = p.sl2 * reinterpret_cast<volatile float*>(gb + G::kQfacOff)[buf * TILES * kTile + (in ? rt : 0)];
                    // the keys of group g (32 keys) this row sees, as bits
                    auto visible = [&](int g) -> uint32_t {
                        const int a0 = p0 + 32 * g - w.q.base;   // tree index of the first key
                        uint32_t v;
                        if (a0 <= -32) {
                            v = ~0u;
                        } else if (a0 < 0) {
                            v = (am[0] << -a0) | ((1u << -a0) - 1u);
                        } else {
                            const int wd = a0 >> 5;
                            const uint32_t lo = wd < 4 ? am[wd] : 0u, hi = wd + 1 < 4 ? am[wd + 1] : 0u;
                            v = __funnelshift_r(lo, hi, a0 & 31);
                        }
                        const int lim = min(np * kBlock, w.q.L - p0) - 32 * g;
                        if (lim < 32) v &= lim <= 0 ? 0u : (1u << lim) - 1u;
                        return v;
                    };
                    // ---- the largest scaled score of this half, then of both
                    float mx = -INFINITY;
                    uint32_t vis[2] = {~0u, ~0u};
                    if (masked) {
                        vis[0] = visible(2 * half);
                        vis[1] = visible(2 * half + 1);
                    }
                    if (!masked && sl2 >= 0.f) {
                        float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            a[k & 3] = max3(a[k & 3], __uint_as_float(sr[0][k]), __uint_as_float(sr[1][k]));
                        mx = fmaxf(max3(a[0], a[1], a[2]), a[3]) * sl2;
                    } else {
#pragma unroll
                        for (int g = 0; g < 2; ++g)
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                mx = fmaxf(mx, (vis[g] >> k) & 1u ? __uint_as_float(sr[g][k]) * sl2 : -INFINITY);
                    }
                    maxima[half * kTile] = mx;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(max_bar);
                    ok = wait_warp(max_bar, met, misc);
                    if (!ok) break;
                    met ^= 1u;
                    mx = fmaxf(mx, maxima[(1 - half) * kTile]);
                    // ---- the reference moves only when it lags by more than 2^8; what
                    // has been accumulated is then scaled down in place
                    const bool move = in && mx > m_ref + kMaxLag;      // (m_ref is -inf at first)
                    if (__any_sync(kFull, move)) {
                        const float alpha = move ? ex2(m_ref - mx) : 1.f;    // 0 while nothing was seen
                        if (move) m_ref = mx;
                        l *= alpha;
#pragma unroll 1
                        for (int c0 = first ? D : half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 16) {
                            uint32_t o[16];
                            umma::tmem_ld16(tO0 + (uint32_t)(128 * st + c0), o);
                            umma::tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                            umma::tmem_st16(tO0 + (uint32_t)(128 * st + c0), o);
                        }
                    }
                    // ---- weights, in place of the scores
                    const float nm = (m_ref == -INFINITY ? 0.f : -m_ref) + (FP8 ? kBiasF16 : 0.f);
                    const u64 sl22 = pack2(sl2, sl2), nm2 = pack2(nm, nm);
                    u64 ls[2] = {0ull, 0ull};
                    float lr[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
                    // all: no key is masked; fused: see kFusedTo
                    auto weigh = [&](auto all, auto fused) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            uint32_t hi[16], lo[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float w0, w1;
                                if (decltype(fused)::value) {
                                    unpack2(fma2(pack2(__uint_as_float(sr[g][2 * e]), __uint_as_float(sr[g][2 * e + 1])),
                                                 sl22, nm2),
                                            w0, w1);
                                } else {
                                    w0 = __fadd_rn(__fmul_rn(__uint_as_float(sr[g][2 * e]), sl2), nm);
                                    w1 = __fadd_rn(__fmul_rn(__uint_as_float(sr[g][2 * e + 1]), sl2), nm);
                                }
                                w0 = ex2(w0);
                                w1 = ex2(w1);
                                if (!decltype(all)::value) {
                                    w0 = (vis[g] >> (2 * e)) & 1u ? w0 : 0.f;
                                    w1 = (vis[g] >> (2 * e + 1)) & 1u ? w1 : 0.f;
                                }
                                hi[e] = FP8 ? pack_f16x2(w0, w1) : pack_bf16x2(w0, w1);
                                if (LOW) lo[e] = pack_bf16x2(w0 - bf16_lo(hi[e]), w1 - bf16_hi(hi[e]));
                                if (!FP8 && !LOW) add_bf16x2(lr[e & 1][0], lr[e & 1][1], hi[e]);
                                else ls[e & 1] = add2(ls[e & 1], pack2(w0, w1));
                            }
                            umma::tmem_st16(tS + (uint32_t)(32 * g), hi);
                            if (LOW) umma::tmem_st16(tS + (uint32_t)(32 * g + 16), lo);
                        }
                    };
                    if (__any_sync(kFull, fabsf(nm) > kFusedTo)) weigh(std::false_type(), std::false_type());
                    else if (masked) weigh(std::false_type(), std::true_type());
                    else weigh(std::true_type(), std::true_type());
                    float l0, l1;
                    unpack2(add2(ls[0], ls[1]), l0, l1);
                    l += (l0 + l1) + ((lr[0][0] + lr[0][1]) + (lr[1][0] + lr[1][1]));
                    first = false;
                    umma::tmem_wait_st();
                    umma::fence_before_sync();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(G::B_PFULL + st));
                ++pc;
            }
            if (!ok) break;
            // ---- the segment's result
            ok = wait_warp(bar(G::B_OFULL), (uint32_t)(seg & 1), misc);
            if (!ok) break;
            umma::fence_after_sync();
            // a padding node sees nothing
            const bool pad = in && ((padw[buf * 4 + (node >> 5)] >> (node & 31)) & 1u);
            if (pad) {
                m_ref = -INFINITY;
                l = 0.f;
            }
            // the halves' sums, and (TILES == 1) the streams' accumulators with their weights
            float a0 = 1.f, a1 = 0.f;
            volatile float* ml = reinterpret_cast<volatile float*>(gb + G::kMlOff) + 2 * r;
            ml[(st * 2 + half) * 2 * kTile] = m_ref;
            ml[(st * 2 + half) * 2 * kTile + 1] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(G::B_ML));
            ok = wait_warp(bar(G::B_ML), (uint32_t)(seg & 1), misc);
            if (!ok) break;
            if (TILES == 2) {
                l = ml[st * 4 * kTile + 1] + ml[(st * 2 + 1) * 2 * kTile + 1];
            } else {
                const float m0 = ml[0], l0 = ml[1] + ml[2 * kTile + 1];
                const float m1 = ml[4 * kTile], l1 = ml[4 * kTile + 1] + ml[6 * kTile + 1];
                const float mm = fmaxf(m0, m1);
                a0 = m0 == -INFINITY ? 0.f : ex2(m0 - mm);
                a1 = m1 == -INFINITY ? 0.f : ex2(m1 - mm);
                m_ref = mm;
                l = l0 * a0 + l1 * a1;
            }
            if (warp_live && !idle) {
                const bool whole = w.j == 0 && w.np == w.q.nb;
                const int g = r0 + rt - node * p.G;
                const size_t orow = ((size_t)(w.q.t0 + node) * p.Hq + (size_t)w.h * p.G + (in ? g : 0)) * D;
                const size_t prow = (((size_t)blockIdx.x * 2 + (w.j == 0 ? 1 : 0)) * (TILES * kTile) + rt);
                const float inv = l == 0.f ? 0.f : v_scale / l;
                // drafted V rows that were zeroed for their infinities or NaN
                uint32_t back[4] = {0u, 0u, 0u, 0u};
                bool any_back = false;
                if (w.drafted(nc - 1)) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t b = 0u;
                        for (int q = 0; q < G::kPrepWarps; ++q) b |= badw[(buf * G::kPrepWarps + q) * 4 + k];
                        back[k] = in && !pad ? b & am[k] : 0u;
                        any_back = any_back || back[k] != 0u;
                    }
                }
                // this warp's share of the output's columns, 16 at a time
                constexpr int kShare = D / (TILES == 1 ? 4 : 2);
                const int c_lo = (TILES == 1 ? st * 2 + half : half) * kShare;
#pragma unroll 1
                for (int c0 = c_lo; c0 < c_lo + kShare; c0 += 16) {
                    uint32_t o[16];
                    umma::tmem_ld16(tO0 + (uint32_t)((TILES == 2 ? 128 * st : 0) + c0), o);
                    umma::tmem_wait_ld();
                    float v[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(o[k]);
                    if (TILES == 1) {
                        if (nc > 1) {            // the second accumulator holds something
                            umma::tmem_ld16(tO0 + (uint32_t)(128 + c0), o);
                            umma::tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) v[k] = v[k] * a0 + __uint_as_float(o[k]) * a1;
                        } else {
#pragma unroll
                            for (int k = 0; k < 16; ++k) v[k] *= a0;
                        }
                    }
                    if (l == 0.f) {
                        const bool lost = whole && in && !pad && sees_any<G::kWords>(w.q, am);
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] = lost ? __uint_as_float(0x7fffffffu) : 0.f;
                    }
                    if (any_back) {
#pragma unroll 1
                        for (int k4 = 0; k4 < 4; ++k4) {
                            for (uint32_t b = k4 == 0 ? back[0] : k4 == 1 ? back[1] : k4 == 2 ? back[2] : back[3];
                                 b != 0u; b &= b - 1u) {
                                const int pos = w.q.base + 32 * k4 + __ffs(b) - 1;
                                const int blk = __ldg(p.bt + (size_t)w.s * p.max_blocks + pos / kBlock);
                                if (blk < 0 || blk >= p.num_blocks) continue;
                                const size_t at = (((size_t)blk * p.Hkv + w.h) * kBlock + pos % kBlock) * D + c0;
#pragma unroll
                                for (int k = 0; k < 16; ++k) {
                                    if (FP8) {
                                        if ((p.v_cache[at + k] & 0x7fu) == 0x7fu) v[k] = __uint_as_float(0x7fffffffu);
                                    } else {
                                        const float z = __uint_as_float(
                                            (uint32_t) reinterpret_cast<const uint16_t*>(p.v_cache)[at + k] << 16);
                                        if (!(fabsf(z) < INFINITY)) v[k] += z;
                                    }
                                }
                            }
                        }
                    }
                    if (!in) continue;
                    if (whole) {
                        if (p.out_f32) {
                            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + orow + c0);
#pragma unroll
                            for (int k = 0; k < 16; k += 4)
                                dst[k / 4] = make_float4(v[k] * inv, v[k + 1] * inv, v[k + 2] * inv, v[k + 3] * inv);
                        } else {
                            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + orow + c0);
#pragma unroll
                            for (int k = 0; k < 16; k += 8)
                                dst[k / 8] = make_uint4(pack_bf16x2(v[k] * inv, v[k + 1] * inv),
                                                        pack_bf16x2(v[k + 2] * inv, v[k + 3] * inv),
                                                        pack_bf16x2(v[k + 4] * inv, v[k + 5] * inv),
                                                        pack_bf16x2(v[k + 6] * inv, v[k + 7] * inv));
                        }
                    } else {
                        float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + c0);
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            dst[k / 4] = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    }
                }
                if (in && !whole && half == 0 && (TILES == 2 || st == 0)) p.part_ml[prow] = make_float2(m_ref, l);
                if (tid == 0 && w.j == 0 && !whole) {
                    // the CTA with the first pages says where the partials are
                    const int last = (int)(((long long)flat + w.q.nb - 1) / misc[M_Q]);
                    p.meta[blockIdx.x] = make_int4(w.s, w.h, last - cta + 1, min(rows, TILES * kTile));
                }
            }
            flat += w.np + kExtraPages;
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(G::B_OFREE + buf));
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == G::kMmaWarp) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------- merge

// The partials of one kernel's CTAs, R rows each.
struct Partials {
    const float* o;
    const float2* ml;
    const int4* meta;
    int ctas, nctas, R;
};

// CTA (x, y): rows 8 y .. 8 y + 7 of the pair whose first partial CTA x of the
// kernel for many (a) or few rows (b) wrote; one warp per row, the partials in
// CTA order.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_tree_merge_kernel(const TreeParams p, const Partials a,
                                                                            const Partials b)
{
    pdl_wait();
    pdl_launch_dependents();
    const bool second = (int)blockIdx.x >= a.ctas;
    const Partials s = second ? b : a;
    const int x = blockIdx.x - (second ? a.ctas : 0);
    const int4 meta = s.meta[x];
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
    const int parts = meta.z;
    if (parts <= 1 || row >= meta.w) return;
    constexpr int V = D / 32;
    // partial i of the pair: the first CTA's second slot, then the first slots
    auto slot = [&](int i) { return ((size_t)(x + i) * 2 + (i == 0 ? 1 : 0)) * s.R + row; };
    float M = -INFINITY;
    for (int i = lane; i < parts; i += 32) M = fmaxf(M, s.ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    float acc[V], l = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float2 ml = s.ml[slot(i)];
        const float* src = s.o + slot(i) * D + lane * V;
        float o[V];
        if constexpr (V == 4) {
            const float4 t = *reinterpret_cast<const float4*>(src);
            o[0] = t.x; o[1] = t.y; o[2] = t.z; o[3] = t.w;
        } else {
            const float2 t = *reinterpret_cast<const float2*>(src);
            o[0] = t.x; o[1] = t.y;
        }
        // a partial that saw nothing weighs nothing (its maximum is -inf)
        const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
        l += ml.y * w;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += o[k] * w;
    }
    const float inv = l == 0.f ? 0.f : p.v_scale / l;
    const int r = x / s.nctas * s.R + row, node = row_node(p, r), g = r - node * p.G;
    int t0, n, bad;
    tree_span(p.starts, meta.x, p.total, p.max_nodes, t0, n, bad);
    const size_t at = ((size_t)(t0 + node) * p.Hq + (size_t)meta.y * p.G + g) * D + lane * V;
    float none = 0.f;                            // the result of a row without weight
    if (l == 0.f) {
        const SeqInfo q = seq_info(p, meta.x, 0, false);
        bool any = q.base > 0 && tree_parent(p.parents, t0, node, nullptr) != KV_TREE_PAD;
        if (q.base == 0)
            for (int a = node; a >= 0 && !any;) {
                const int up = tree_parent(p.parents, t0, a, nullptr);
                any = up != KV_TREE_PAD && a < q.L;
                a = up;
            }
        if (any) none = __uint_as_float(0x7fffffffu);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = l == 0.f ? none : acc[k] * inv;
    if (p.out_f32) {
        float* dst = static_cast<float*>(p.out) + at;
        if constexpr (V == 4) *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        else *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
    } else {
        uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
        if constexpr (V == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
        else
            *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0], acc[1]);
    }
}

// -------------------------------------------------------------------- host

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

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// The kernels a shape may need, their tiles and teams, and the workspace:
// partial outputs, their (max, sum) and the tables of both.
struct TreePlan {
    bool few, many;             // sequences of up to / above kSmallRows rows
    int few_rows, few_ctas;
    int tiles, teams, nctas;
    size_t few_o, few_ml, few_meta, many_o, many_ml, many_meta, total;
};

TreePlan tree_plan(int max_nodes, int G, int D)
{
    TreePlan t;
    const int rows = max_nodes * G, sms = num_sms_current();
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += up256(bytes);
        return here;
    };
    t.few = G <= kSmallRows;
    t.many = rows > kSmallRows;
    t.few_rows = tree_small_rows(std::min(rows, kSmallRows));
    t.few_ctas = t.few ? sms : 0;
    const size_t few_slots = (size_t)t.few_ctas * 2 * t.few_rows;
    t.few_o = take(few_slots * D * sizeof(float));
    t.few_ml = take(few_slots * sizeof(float2));
    t.few_meta = take((size_t)t.few_ctas * sizeof(int4));
    t.tiles = rows > kTile ? 2 : 1;
    t.teams = (rows + t.tiles * kTile - 1) / (t.tiles * kTile);
    t.nctas = t.many ? std::max(1, sms / t.teams) : 0;
    // (room for a CTA per SM, also where the teams leave some SMs out: what serves
    // max_nodes nodes then serves fewer too)
    const size_t many_ctas = t.many ? (size_t)std::max(sms, t.teams) : 0;
    const size_t many_slots = many_ctas * 2 * t.tiles * kTile;
    t.many_o = take(many_slots * D * sizeof(float));
    t.many_ml = take(many_slots * sizeof(float2));
    t.many_meta = take(many_ctas * sizeof(int4));
    t.total = at;
    return t;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, unsigned block, size_t smem,
                       cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int kMaxDevices = 64;
std::mutex g_tree_mu;

template <int D, bool FP8, int TILES, bool LOW>
cudaError_t launch_many(const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, cudaStream_t st)
{
    using G = Geo<D, FP8, TILES>;
    static bool ready[kMaxDevices] = {};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(g_tree_mu);
        if (!ready[dev]) {
            if (cudaError_t e = cudaFuncSetAttribute(paged_tree_kernel<D, FP8, TILES, LOW>,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem))
                return e;
            ready[dev] = true;
        }
    }
    return launch_pdl(paged_tree_kernel<D, FP8, TILES, LOW>, dim3((unsigned)(p.teams * p.nctas)), G::kThreads,
                      G::kSmem, st, mk, mv, p);
}

template <int D, int TILES>
cudaError_t launch_many(const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, bool fp8,
                        cudaStream_t st)
{
    if (fp8) return launch_many<D, true, TILES, false>(mk, mv, p, st);
    return p.out_f32 ? launch_many<D, false, TILES, true>(mk, mv, p, st)
                     : launch_many<D, false, TILES, false>(mk, mv, p, st);
}

}  // namespace

int tree_read_error(unsigned* flags, long long* detail) { return g_launched.take_error(g_tree_err, flags, detail); }

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
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KV_ERR_CUDA;
    *bytes = tree_plan(max_nodes, num_q_heads / num_kv_heads, head_dim).total;
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
    // flat work indices and tensor-map rows must fit in int32
    if (((long long)max_blocks_per_seq + kExtraPages) * num_seqs * num_kv_heads >= INT_MAX ||
        (long long)num_blocks * num_kv_heads >= INT_MAX ||
        (long long)max_blocks_per_seq * kBlock >= INT_MAX ||
        (long long)total_nodes * num_q_heads >= INT_MAX)
        return KV_ERR_UNSUPPORTED;
    const TreePlan t = tree_plan(max_nodes, num_q_heads / num_kv_heads, head_dim);
    if (workspace_bytes < t.total) return KV_ERR_INVALID_ARG;
    CUtensorMap mk, mv;
    if (int rc = cache_tensor_map(&mk, k_cache, head_dim, fp8, num_blocks, num_kv_heads)) return rc;
    if (int rc = cache_tensor_map(&mv, v_cache, head_dim, fp8, num_blocks, num_kv_heads)) return rc;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
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
    p.g_magic = p.G == 1 ? 0u : 0xffffffffu / (uint32_t)p.G + 1u;
    p.min_q = kMinPages;
    p.sl2 = scale * 1.4426950408889634f * (fp8 ? k_scale : 1.f);
    p.v_scale = fp8 ? v_scale : 1.f;
    p.out_f32 = out_dtype == KV_DTYPE_F32;
    p.test_stall = test_stall_cycles();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    Partials few = {}, many = {};
    g_launched.note();
    if (t.few) {
        p.part_o = reinterpret_cast<float*>(ws + t.few_o);
        p.part_ml = reinterpret_cast<float2*>(ws + t.few_ml);
        p.meta = reinterpret_cast<int4*>(ws + t.few_meta);
        p.nctas = t.few_ctas;
        p.teams = 1;
        p.rows_above = 0;
        p.rows_to = kSmallRows;
        p.tidy = 1;
        if (tree_small_launch(mk, mv, p, head_dim, fp8, t.few_rows, st) != cudaSuccess) return KV_ERR_CUDA;
        few = {p.part_o, p.part_ml, p.meta, t.few_ctas, t.few_ctas, t.few_rows};
    }
    if (t.many) {
        p.part_o = reinterpret_cast<float*>(ws + t.many_o);
        p.part_ml = reinterpret_cast<float2*>(ws + t.many_ml);
        p.meta = reinterpret_cast<int4*>(ws + t.many_meta);
        p.nctas = t.nctas;
        p.teams = t.teams;
        p.rows_above = t.few ? kSmallRows : 0;
        p.rows_to = INT_MAX;
        p.tidy = !t.few;
        cudaError_t err;
        if (head_dim == 128)
            err = t.tiles == 1 ? launch_many<128, 1>(mk, mv, p, fp8, st) : launch_many<128, 2>(mk, mv, p, fp8, st);
        else
            err = t.tiles == 1 ? launch_many<64, 1>(mk, mv, p, fp8, st) : launch_many<64, 2>(mk, mv, p, fp8, st);
        if (err != cudaSuccess) return KV_ERR_CUDA;
        many = {p.part_o, p.part_ml, p.meta, t.teams * t.nctas, t.nctas, t.tiles * kTile};
    }
    const int rows = std::max(t.few ? std::min(max_nodes * p.G, kSmallRows) : 0,
                              t.many ? std::min(max_nodes * p.G, t.tiles * kTile) : 0);
    const dim3 grid((unsigned)(many.ctas + few.ctas), (unsigned)((rows + kMergeWarps - 1) / kMergeWarps));
    const cudaError_t err =
        head_dim == 128 ? launch_pdl(paged_tree_merge_kernel<128>, grid, kMergeWarps * 32, 0, st, p, many, few)
                        : launch_pdl(paged_tree_merge_kernel<64>, grid, kMergeWarps * 32, 0, st, p, many, few);
    return err == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}
