// paged_tree_attention for sequences of at most 64 query rows per KV head (nodes
// times heads per KV head): small trees, and single tokens.
//
// The mathematics is paged_tree.cu's; the products are the other way round.  A
// tcgen05.mma of M = 128 takes ~64 clocks whatever its N up to 128 (measured),
// so with the queries as M, 32 rows would cost what 128 do.  Here the 128 keys of
// a chunk, and then the head's dimensions, are M, and the rows are N:
//     S^T = K Q^T   (128 keys x N rows, K as it lies in the ring),
//     O^T += V^T P^T   (head_dim x N, V as it lies in the ring, P through shared
//                       memory; its high and low parts are N columns each of ONE
//                       product, added at the end: the low part costs nothing).
// 16 products, ~1030 clocks, for 128 keys, whose bf16 K and V take ~2450 clocks
// to arrive at 6.8 TB/s over 152 SMs (E4M3: ~1220): HBM is the bound.  Measured:
// 32 x 8192 tokens, 8 nodes x 4 heads, bf16: 167 us (bytes: 159); 4 x 131072: 312
// (316); E4M3, 8 nodes: 121 us, 16 nodes x 4 heads: 166 us (80), where shared memory
// carries ~190 KB a chunk (~1500 clocks: codes, widened V, weights, the MMAs'
// operands), a group's weights take ~2300 clocks, and the query's third part another
// four products.
//
// Scores and products have an MMA thread each: one for both was busy ~2400 clocks a
// chunk, of which the tensor cores 1024, with commits and waits of ~100 clocks (172
// us for 8 nodes, E4M3 124; 16 nodes E4M3 150).
//
// How (the rest as in paged_tree.cu):
//  * One thread per key of a chunk weighs that key for 32 rows, so the
//    exponentials of few rows use all lanes, and a row's sum stays in a register
//    of each lane until the end.  Two groups of four warps: up to 32 rows (N = 32)
//    they take the chunks in turn, each with its own accumulator O^T and
//    references; above (N = 64) each takes 32 rows of every chunk.  The scores run up
//    to four chunks ahead (four S^T buffers).
//  * The reference maximum of a row moves only when a score is more than 2^8
//    above it (the four warps of a group agree on that once per chunk); the first
//    chunk of a segment sets it.  Then, seldom, the columns of O^T and the sums
//    are scaled.
//  * D < 128: the lower lanes of O^T hold the result, the upper ones products of
//    whatever follows V in shared memory, never read.
#include <cuda_runtime.h>

#include <mutex>

#include "cache_map.h"
#include "internal.h"
#include "tree_kernel.cuh"

namespace pkv {

namespace {

template <int D, bool FP8, int N>
struct SmallGeo {
    static constexpr int kD = D;
    static constexpr bool kFp8 = FP8;
    static constexpr bool kSplit = N == 64;                  // the groups split the rows, not the chunks
    static constexpr int kWeighWarps = 8;                    // two groups of four
    static constexpr int kCopyWarp = kWeighWarps;            // K; the next V
    static constexpr int kMmaWarp = kCopyWarp + 2;           // scores; the next products
    static constexpr int kPrepWarp = kMmaWarp + 2;           // first of the prep / widening warps
    static constexpr int kPrepWarps = FP8 ? 4 : 1;
    static constexpr int kThreads = (kPrepWarp + kPrepWarps) * 32;
    static constexpr int kBoxes = D / 64;
    static constexpr int kSlot = kBoxes * kRegion;           // K or V of a chunk, 2 bytes each
    static constexpr int kPageBytes = kBlock * D * (FP8 ? 1 : 2);
    static constexpr int kRawSlot = kPages * kBlock * D;     // E4M3 codes of K or V of a chunk
    // columns of P and of an accumulator: the high parts of the rows' weights,
    // then the low parts.  64 rows of an E4M3 cache go without: f16's 11 bits
    // against the cache's 4, and the room goes to the rings.
    static constexpr bool kLow = !(FP8 && N == 64);
    static constexpr int kAccs = kSplit ? 1 : 2;             // accumulators
    static constexpr int kPW = kLow ? 2 * N : N;
    static constexpr int kPBuf = kPW / 64 * kRegion;         // [column group of 64][128 keys][128 B]
    static constexpr int kQBytes = FP8 ? kQueryParts * N * D : kBoxes * N * 128;
    static constexpr int kScale = 128 / D;
    static constexpr int kKSlots = (FP8 ? 4 : 2) * kScale, kVSlots = (FP8 || N == 64 ? 2 : 3) * kScale;
    static constexpr int kRawV = !FP8 ? 0 : (N == 32 ? 3 : 2) * kScale;
    static constexpr int kLoadBytes = FP8 ? kRawSlot : kSlot;
    static constexpr int kQOff = 0;
    static constexpr int kKOff = (kQOff + kQBytes + 1023) / 1024 * 1024;
    static constexpr int kVOff = kKOff + kKSlots * kLoadBytes;
    static constexpr int kPOff = kVOff + kVSlots * kSlot;    // two buffers (behind the ring: see D < 128)
    static constexpr int kRawOff = kPOff + 2 * kPBuf;
    static constexpr int kBarOff = kRawOff + kRawV * kRawSlot;
    static constexpr int kVLoadOff = FP8 ? kRawOff : kVOff;
    // barriers
    static constexpr int kVL = FP8 ? kRawV : kVSlots;
    static constexpr int B_KFULL = 0;                        // + slot: K has landed
    // + chunk % kScoreBars: its scores are there (and its K slot may be refilled)
    static constexpr int kScoreBars = kKSlots > 4 ? kKSlots : 4;
    static constexpr int B_SFULL = B_KFULL + kKSlots;
    static constexpr int B_VFULL = B_SFULL + kScoreBars;     // V, or its codes
    // + slot: it may be refilled (of what the MMAs read: a chunk's products are done)
    static constexpr int B_VEMPTY = B_VFULL + kVL;
    static constexpr int B_VWIDE = B_VEMPTY + kVL;           // (FP8) + slot: widened
    static constexpr int B_VWFREE = B_VWIDE + (FP8 ? kVSlots : 0);
    static constexpr int B_FIX = B_VWFREE + (FP8 ? kVSlots : 0);     // (bf16) + slot: V rows fixed
    using KRing = Ring<kKSlots, B_KFULL, B_SFULL, kScoreBars>;
    using VLoad = Ring<kVL, B_VFULL, B_VEMPTY>;              // what TMA fills, and what the MMAs read
    using VRing = Ring<kVSlots, FP8 ? B_VWIDE : B_VFULL, FP8 ? B_VWFREE : B_VEMPTY>;
    static constexpr int B_QFULL = B_FIX + (FP8 ? 0 : kVSlots);  // Q and the tree of a segment
    static constexpr int B_QFREE = B_QFULL + 1;              // its last scores are computed
    static constexpr int B_SFREE = B_QFREE + 1;              // + buffer (4): the scores have been read
    static constexpr int B_PFULL = B_SFREE + 4;              // + buffer of P: weights written
    static constexpr int B_OFULL = B_PFULL + 2;              // the accumulators are complete
    static constexpr int B_OFREE = B_OFULL + 1;              // + segment & 1: they have been read
    static constexpr int B_JOIN = B_OFREE + 2;               // the groups meet
    static constexpr int B_END = B_JOIN + 1;                 // + MMA warp: all its MMAs are done
    static constexpr int B_STALL = B_END + 2;                // nothing arrives (the test hook)
    static constexpr int kNumBars = B_STALL + 1;
    static constexpr int kMiscOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kWords = N / 32;                    // words of a node's bits (a node has a row)
    static constexpr int kAncOff = kMiscOff + 64;            // [2][N][kWords] words
    static constexpr int kPtrOff = kAncOff + 2 * N * kWords * 4;     // [N] words
    static constexpr int kPadOff = kPtrOff + N * 4;          // [2][4] words
    static constexpr int kBadOff = kPadOff + 32;             // [2][kPrepWarps][4] words
    static constexpr int kQfacOff = kBadOff + 2 * kPrepWarps * 16;   // [2][N] floats (FP8)
    static constexpr int kScOff = kQfacOff + 2 * N * 4;      // [group][row] floats: the scale
    static constexpr int kNrOff = kScOff + 64 * 4;           // [group][row] floats: what is added, -reference
    static constexpr int kRefOff = kNrOff + 64 * 4;          // [group][row] floats: the reference
    static constexpr int kAlphaOff = kRefOff + 64 * 4;       // [group][row] floats
    static constexpr int kWmaxOff = kAlphaOff + 64 * 4;      // [group][4][row] floats: maxima, later sums
    static constexpr int kFacOff = kWmaxOff + 256 * 4;       // [N] float4
    static constexpr int kRowOff = kFacOff + N * 16;         // [N] words: place of a row's result
    static constexpr int kUnsetOff = kRowOff + N * 4;        // [group] words
    static constexpr int kEnd = kUnsetOff + 16;
    static constexpr int kSmem = kEnd + 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    // E4M3: the query's parts are 3 N columns of one product, added by the groups
    // (two parts, 8 nodes x 4 heads of 32 x 8192 tokens: 134 -> 126 us), or, where the
    // groups have no time left (64 rows: 151 -> 159 us), products into the same columns.
    static constexpr bool kSideBySide = FP8 && !kSplit;
    // tensor memory: four S^T buffers, then the accumulators
    static constexpr int kScoreCols = kSideBySide ? kQueryParts * N : N;
    static constexpr uint32_t kColO = 4 * kScoreCols;
    static constexpr uint32_t kTmemCols = kColO + kAccs * kPW <= 256 ? 256 : 512;
    static_assert(kColO + kAccs * kPW <= 512, "tensor memory");
};

// Order-preserving map of floats to ints, NaN above infinity (the one that arithmetic
// gives, whose sign bit is clear).
__device__ __forceinline__ int ordered(float x)
{
    const int b = __float_as_int(x);
    return b >= 0 ? b : b ^ 0x7fffffff;
}

__device__ __forceinline__ float unordered(int b)
{
    return __int_as_float(b >= 0 ? b : b ^ 0x7fffffff);
}

// The larger of two; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Sums over the warp of 32 values a lane: lane l gets the sum of v[l].
__device__ __forceinline__ float column_sums(float (&v)[32], int lane)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < o; ++k) {
            const float keep = up ? v[k + o] : v[k], send = up ? v[k] : v[k + o];
            v[k] = keep + __shfl_xor_sync(kFull, send, o);
        }
    }
    return v[0];
}

template <int D, bool FP8, int N>
__global__ void __launch_bounds__(SmallGeo<D, FP8, N>::kThreads, 1)
paged_tree_small_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const TreeParams p)
{
    using G = SmallGeo<D, FP8, N>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sraw = smem_u32(smem_raw);
    const uint32_t sb = (sraw + 1023u) & ~1023u;
    uint8_t* gb = smem_raw + (sb - sraw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    volatile int* misc = reinterpret_cast<volatile int*>(gb + G::kMiscOff);
    auto bar = [&](int i) -> uint32_t { return sb + (uint32_t)(G::kBarOff + 8 * i); };

    if (tid == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        for (int i = 0; i < G::kKSlots; ++i) mbar_init(bar(G::B_KFULL + i), 1);
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
        for (int i = 0; i < G::kScoreBars; ++i) mbar_init(bar(G::B_SFULL + i), 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar(G::B_PFULL + w), G::kSplit ? G::kWeighWarps : 4);
            mbar_init(bar(G::B_OFREE + w), G::kWeighWarps);
        }
        mbar_init(bar(G::B_OFULL), 1);
        mbar_init(bar(G::B_JOIN), G::kWeighWarps);
        for (int w = 0; w < 2; ++w) mbar_init(bar(G::B_END + w), 1);
        for (int i = 0; i < 4; ++i) mbar_init(bar(G::B_SFREE + i), G::kSplit ? G::kWeighWarps : 4);
        mbar_init(bar(G::B_STALL), 1);
        misc[M_ABORT] = 0;
        misc[M_VISSUED] = 0;
        fence_mbar_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    if (warp == G::kMmaWarp) {
        umma::tmem_alloc(sb + G::kMiscOff + 4 * M_TMEM, G::kTmemCols);
        umma::tmem_relinquish();
    }
    if (warp == G::kCopyWarp) cut_work(p, misc, 0, cta, p.tidy && cta == 0, lane);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = (uint32_t)misc[M_TMEM];

    if (warp == G::kCopyWarp) {
        copy_role<G, 0>(p, tm_k, tm_v, sb, misc, 0, lane);
    } else if (warp == G::kCopyWarp + 1) {
        copy_role<G, 1>(p, tm_k, tm_v, sb, misc, 0, lane);
    } else if (warp == G::kMmaWarp) {
        // ------------------------------------------------------------- scores
        if (lane == 0) {
            const uint64_t qdesc = FP8 ? code_desc<D>(sb + G::kQOff) : umma::smem_desc_sw128(sb + G::kQOff, 16, 1024);
            const uint64_t kdesc = FP8 ? code_desc<D>(sb + G::kKOff) : umma::smem_desc_sw128(sb + G::kKOff, 16, 1024);
            constexpr uint32_t idesc_s = FP8 ? umma::idesc_f8_f32(128, G::kScoreCols, false, true)
                                             : umma::idesc_bf16_f32(128, N, false, false);
            using KR = typename G::KRing;
            int g = 0;                           // chunk of the CTA
            bool ok = true;
            if (p.test_stall > 0 && misc[M_CNT] > 0 &&
                !mbar_wait_bounded(bar(G::B_STALL), 0u, p.test_stall)) {
                misc[M_ABORT] = 1;
                raise_flag(&g_tree_err, KV_DEVERR_PIPELINE_TIMEOUT, blockIdx.x);
                ok = false;
            }
            for (Walk w(p, misc, 0); ok && w.more(); w.next(p, 0)) {
                const int nc = w.chunks();
                ok = wait_bar(bar(G::B_QFULL), (uint32_t)(w.seg & 1), misc);
                for (int c = 0; ok && c < nc; ++c, ++g) {
                    // the buffer was read for chunk g - 4
                    if (g >= 4) ok = wait_bar(bar(G::B_SFREE + (g & 3)), (uint32_t)((g >> 2) - 1) & 1u, misc);
                    ok = ok && wait_bar(bar(KR::full(g)), KR::parity(g), misc);
                    if (!ok) break;
                    umma::fence_after_sync();
                    const uint64_t kd = kdesc + (uint64_t)((KR::slot(g) * G::kLoadBytes) >> 4);
                    const uint32_t d = tmem + (uint32_t)(G::kScoreCols * (g & 3));
                    if constexpr (FP8) {
#pragma unroll
                        for (int part = 0; part < (G::kSideBySide ? 1 : kQueryParts); ++part)
#pragma unroll
                            for (int kk = 0; kk < D / 32; ++kk)
                                umma::mma_f8_ss(d, kd + (uint64_t)((kk * 32) >> 4),
                                                qdesc + (uint64_t)((part * N * D + kk * 32) >> 4), idesc_s,
                                                part + kk > 0);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            umma::mma_bf16_ss(d, kd + (uint64_t)(((kk >> 2) * kRegion + (kk & 3) * 32) >> 4),
                                              qdesc + (uint64_t)(((kk >> 2) * N * 128 + (kk & 3) * 32) >> 4),
                                              idesc_s, kk > 0);
                    }
                    // (one commit for the scores and the slot of K: each takes this
                    // thread ~100 clocks)
                    umma::commit(bar(KR::free(g)));
                    if (c + 1 == nc) umma::commit(bar(G::B_QFREE));
                }
            }
            // every MMA issued by this thread is complete before the CTA ends
            umma::commit(bar(G::B_END));
            mbar_wait_bounded(bar(G::B_END), 0u, kWaitLimit);
        }
        __syncwarp();
    } else if (warp == G::kMmaWarp + 1) {
        // ----------------------------------------------------------- products
        if (lane == 0) {
            const uint64_t vdesc = umma::smem_desc_sw128(sb + G::kVOff, kRegion, 1024);
            const uint64_t pdesc = umma::smem_desc_sw128(sb + G::kPOff, kRegion, 1024);
            constexpr uint32_t idesc_pv = FP8 ? umma::idesc_f16_f32(128, G::kPW, true, true)
                                              : umma::idesc_bf16_f32(128, G::kPW, true, true);
            using VR = typename G::VRing;
            uint32_t fix_parity = 0;             // bit slot: parity of its next fix
            int g = 0;                           // chunk of the CTA
            bool ok = true;
            for (Walk w(p, misc, 0); ok && w.more(); w.next(p, 0)) {
                const int nc = w.chunks(), seg = w.seg;
                for (int c = 0; ok && c < nc; ++c, ++g) {
                    const int vs = VR::slot(g), pbuf = g & 1;
                    // what is usually there comes first, the weights last
                    ok = wait_bar(bar(VR::full(g)), VR::parity(g), misc);
                    if (ok && !FP8 && w.drafted(c)) {
                        ok = wait_bar(bar(G::B_FIX + vs), (fix_parity >> vs) & 1u, misc);
                        fix_parity ^= 1u << vs;
                    }
                    // the accumulators of the segment before have been read
                    if (ok && c < G::kAccs && seg > 0)
                        ok = wait_bar(bar(G::B_OFREE + ((seg - 1) & 1)), (uint32_t)(((seg - 1) >> 1) & 1), misc);
                    ok = ok && wait_bar(bar(G::B_PFULL + pbuf), (uint32_t)((g >> 1) & 1), misc);
                    if (!ok) break;
                    umma::fence_after_sync();
                    const uint64_t vd = vdesc + (uint64_t)((vs * G::kSlot) >> 4);
                    const uint64_t pd = pdesc + (uint64_t)((pbuf * G::kPBuf) >> 4);
                    const int np = w.chunk_pages(c);
                    auto page = [&](int kk) {
                        umma::mma_bf16_ss(tmem + G::kColO + (uint32_t)(G::kSplit ? 0 : pbuf * G::kPW),
                                          vd + (uint64_t)((kk * kBlock * 128) >> 4),
                                          pd + (uint64_t)((kk * kBlock * 128) >> 4), idesc_pv,
                                          !(c < G::kAccs && kk == 0));
                    };
                    if (np == kPages) {
#pragma unroll
                        for (int kk = 0; kk < kPages; ++kk) page(kk);
                    } else {
#pragma unroll 1
                        for (int kk = 0; kk < np; ++kk) page(kk);
                    }
                    umma::commit(bar(VR::free(g)));      // and the buffer of P
                    if (c + 1 == nc) umma::commit(bar(G::B_OFULL));
                }
            }
            umma::commit(bar(G::B_END + 1));
            mbar_wait_bounded(bar(G::B_END + 1), 0u, kWaitLimit);
        }
        __syncwarp();
    } else if (warp >= G::kPrepWarp) {
        // ------------------------- queries, trees, V rows, and widening (E4M3)
        const int pw = warp - G::kPrepWarp;
        int g0 = 0;
        bool ok = true;
        for (Walk w(p, misc, 0); ok && w.more(); w.next(p, 0)) {
            const int seg = w.seg, buf = seg & 1;
            // the segment's entry of the tree tables was last read two segments ago
            if (seg >= 2) ok = wait_warp(bar(G::B_OFREE + buf), (uint32_t)(((seg - 2) >> 1) & 1), misc);
            if (ok && seg >= 1) ok = wait_warp(bar(G::B_QFREE), (uint32_t)((seg - 1) & 1), misc);
            if (!ok) break;
            volatile uint32_t* badw = reinterpret_cast<volatile uint32_t*>(gb + G::kBadOff);
            if (lane < 4) badw[(buf * G::kPrepWarps + pw) * 4 + lane] = 0u;
            const int rows = w.q.n * p.G;        // <= N
            constexpr int C = D / 8, RI = 32 / C;    // 16-byte chunks of a row, rows of an instruction
            const int c = lane % C;
            for (int rb = pw * RI; rb < rows; rb += G::kPrepWarps * RI) {
                const int r = rb + lane / C, rc = min(r, rows - 1);
                const int node = row_node(p, rc), gq = rc - node * p.G;
                const uint16_t* src =
                    p.q + ((size_t)(w.q.t0 + node) * p.Hq + (size_t)w.h * p.G + gq) * D + 8 * c;
                if (!FP8) {
                    const uint32_t dst = sb + (uint32_t)(G::kQOff + (c >> 3) * N * 128) + region_off(rc, c & 7);
                    if (r < rows) cp_async16(dst, src);
                } else {
                    float up;
                    uint2 parts[kQueryParts];
                    query_e5m2<D>(__ldg(reinterpret_cast<const uint4*>(src)), parts, up);
                    if (r < rows) {
                        const uint32_t at = sb + (uint32_t)G::kQOff + code_off<D>(rc, c);
#pragma unroll
                        for (int part = 0; part < kQueryParts; ++part) sts64(at + (uint32_t)(part * N * D), parts[part]);
                        if (c == 0) reinterpret_cast<volatile float*>(gb + G::kQfacOff)[buf * N + r] = up;
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
            g0 += w.chunks();
        }
        if (!FP8) cp_async_wait_all();
    } else {
        // ------------------------------------------------- weights and output
        const int grp = warp >> 2, key = tid & 127, wq = warp & 3;
        constexpr int R = 32;                    // rows that a group weighs
        const int row0 = G::kSplit ? R * grp : 0;        // the group's first row
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        // the group's columns of its accumulator; the low parts are N further on
        const uint32_t tO = lanes + G::kColO + (uint32_t)(G::kSplit ? row0 : grp * G::kPW);
        float* sc = reinterpret_cast<float*>(gb + G::kScOff) + grp * R;
        float* nr = reinterpret_cast<float*>(gb + G::kNrOff) + grp * R;
        float* ref = reinterpret_cast<float*>(gb + G::kRefOff) + grp * R;
        float* alphas = reinterpret_cast<float*>(gb + G::kAlphaOff) + grp * R;
        float* wmax = reinterpret_cast<float*>(gb + G::kWmaxOff) + grp * 4 * R;
        volatile int* unset = reinterpret_cast<volatile int*>(gb + G::kUnsetOff) + grp;
        if (p.tidy) zero_empty(p, D, cta, p.nctas, tid, G::kWeighWarps * 32);
        if (tid == 0) p.meta[cta] = make_int4(0, 0, 0, 0);
        int joins = 0, g0 = 0, flat = misc[M_B0];
        bool ok = true;
        // The group's four warps meet: is `x` true anywhere?  Every warp comes to every
        // meeting, also one whose waits have run out, which the others learn there.
        auto meet = [&](bool x) -> bool {
            int r;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\t"
                "barrier.cta.red.or.pred q, %1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
                : "=r"(r)
                : "r"(1 + grp), "r"(x ? 1 : 0)
                : "memory");
            return r != 0;
        };
        auto join = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(G::B_JOIN));
            const bool r = wait_warp(bar(G::B_JOIN), (uint32_t)(joins & 1), misc);
            ++joins;
            return r;
        };
        for (Walk w(p, misc, 0); ok && w.more(); w.next(p, 0)) {
            const int seg = w.seg, buf = seg & 1, nc = w.chunks();
            const int rows = w.q.n * p.G;
            const uint32_t* anc = reinterpret_cast<const uint32_t*>(gb + G::kAncOff) + buf * N * G::kWords;
            const volatile uint32_t* padw = reinterpret_cast<const volatile uint32_t*>(gb + G::kPadOff) + buf * 4;
            const int plain = w.plain_chunks();
            float l[R];                          // each row's sum over this thread's keys
#pragma unroll
            for (int k = 0; k < R; ++k) l[k] = 0.f;
            bool first = true, pending = false;  // pending: a row has no reference yet
            bool wide = false;                   // a row's is above kFusedTo
            for (int c = G::kSplit ? 0 : (g0 ^ grp) & 1; c < nc; c += G::kSplit ? 1 : 2) {
                const int g = g0 + c;
                // the scores; and the buffer of P: the products of the chunk before last
                // are done, which groups that take every chunk wait for here, others,
                // whose own last chunk that was, when they need it.  (A wait that runs out
                // is told at the next meeting; nothing is written then.)
                auto buffer_free = [&]() -> bool {
                    return g < 2 || wait_bar(bar(G::VRing::free(g - 2)), G::VRing::free_parity(g - 2), misc);
                };
                ok = __all_sync(kFull, ok && wait_bar(bar(G::KRing::free(g)), G::KRing::free_parity(g), misc) &&
                                           (!G::kSplit || buffer_free()));
                if (first) {
                    // the rows' scale and reference: none yet for rows that see
                    // something, and never a weight for the others
                    if (wq == 0) {
                        const int r = row0 + lane, nd = r < rows ? row_node(p, r) : 0;
                        const bool live = r < rows && !((padw[nd >> 5] >> (nd & 31)) & 1u);
                        const float f = FP8 && live ? reinterpret_cast<volatile float*>(gb + G::kQfacOff)[buf * N + r] : 1.f;
                        sc[lane] = live ? p.sl2 * f : 0.f;
                        nr[lane] = live ? 0.f : -INFINITY;
                        ref[lane] = -INFINITY;
                        const bool any = __any_sync(kFull, live);
                        if (lane == 0) *unset = any;
                    }
                    if (meet(!ok)) ok = false;
                    pending = *unset != 0;
                }
                umma::fence_after_sync();
                const uint32_t tS = lanes + (uint32_t)(G::kScoreCols * (g & 3) + row0);
                const bool masked = c >= plain;          // (for the whole chunk)
                // the rows that see this key, as bits
                uint32_t vis = ~0u;
                bool there = true;                       // is the key in one of the chunk's pages?
                if (masked) {
                    const int pos = (w.j + c * kPages) * kBlock + key;
                    there = key < w.chunk_pages(c) * kBlock;
                    vis = there && pos < w.q.L ? ~0u : 0u;
                    if (pos >= w.q.base && vis) {
                        const int a = pos - w.q.base;
                        vis = 0u;
                        for (int r = row0; r < min(rows, row0 + R); ++r)
                            vis |= ((anc[row_node(p, r) * G::kWords + (a >> 5)] >> (a & 31)) & 1u) << (r - row0);
                    }
                }
                // 16 rows' scores as the products left them
                auto load16 = [&](int k0, float* x) {
                    uint32_t(&a)[16] = *reinterpret_cast<uint32_t(*)[16]>(x);
                    umma::tmem_ld16(tS + (uint32_t)k0, a);
                    if (G::kSideBySide) {
                        uint32_t b[16], c[16];
                        umma::tmem_ld16(tS + (uint32_t)(N + k0), b);
                        umma::tmem_ld16(tS + (uint32_t)(2 * N + k0), c);
                        umma::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) x[k] += __uint_as_float(b[k]) + __uint_as_float(c[k]);
                    } else {
                        umma::tmem_wait_ld();
                    }
                };
                // the scores relative to the references, in log2 units
                float t[R];
                auto load = [&]() {
                    if (G::kSideBySide) {
                        load16(0, t);
                        load16(16, t + 16);
                    } else {
                        umma::tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[R]>(&t[0]));
                        umma::tmem_wait_ld();
                    }
                    if (!wide) {
#pragma unroll
                        for (int k = 0; k < R; k += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(sc + k);
                            const float4 n = *reinterpret_cast<const float4*>(nr + k);
                            unpack2(fma2(pack2(t[k], t[k + 1]), pack2(f.x, f.y), pack2(n.x, n.y)), t[k], t[k + 1]);
                            unpack2(fma2(pack2(t[k + 2], t[k + 3]), pack2(f.z, f.w), pack2(n.z, n.w)), t[k + 2], t[k + 3]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < R; k += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(sc + k);
                            const float4 n = *reinterpret_cast<const float4*>(nr + k);
                            t[k] = __fadd_rn(__fmul_rn(t[k], f.x), n.x);
                            t[k + 1] = __fadd_rn(__fmul_rn(t[k + 1], f.y), n.y);
                            t[k + 2] = __fadd_rn(__fmul_rn(t[k + 2], f.z), n.z);
                            t[k + 3] = __fadd_rn(__fmul_rn(t[k + 3], f.w), n.w);
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < R; ++k) t[k] = (vis >> k) & 1u ? t[k] : -INFINITY;
                    }
                };
                load();
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < R; k += 2) mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], t[k], t[k + 1]);
                const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                // does any row's reference lag too far behind, or has a wait run out?
                if (meet(!ok || most > kMaxLag + (FP8 ? kBiasF16 : 0.f) || pending)) {
                    if (meet(!ok)) {
                        ok = false;
                        break;
                    }
                    // ---- new references: the largest score of each row in the chunk
                    int best = INT32_MIN;
#pragma unroll 1
                    for (int k0 = 0; k0 < R; k0 += 16) {
                        float x[16];
                        load16(k0, x);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            x[k] = (vis >> (k0 + k)) & 1u ? __fmul_rn(x[k], sc[k0 + k]) : -INFINITY;
                            const int m = __reduce_max_sync(kFull, ordered(x[k]));
                            if (lane == k0 + k) best = m;
                        }
                    }
                    wmax[wq * R + lane] = unordered(best);
                    meet(false);
                    if (wq == 0) {
                        float top = max_nan(max_nan(wmax[lane], wmax[R + lane]),
                                            max_nan(wmax[2 * R + lane], wmax[3 * R + lane]));
                        const float old = ref[lane];
                        const bool live = nr[lane] != -INFINITY;
                        // a row whose first scores hold NaN is NaN whatever its reference: 0
                        if (old == -INFINITY && top != top) top = 0.f;
                        float a = 1.f;
                        if (live && (old == -INFINITY ? top > -INFINITY : top > old + kMaxLag)) {
                            a = old == -INFINITY ? 0.f : ex2(old - top);
                            ref[lane] = top;
                            nr[lane] = (FP8 ? kBiasF16 : 0.f) - top;
                        }
                        alphas[lane] = a;
                        const bool left = __any_sync(kFull, live && ref[lane] == -INFINITY);
                        const bool far = __any_sync(kFull, live && ref[lane] != -INFINITY && fabsf(ref[lane]) > kFusedTo);
                        if (lane == 0) *unset = (left ? 1 : 0) + (far ? 2 : 0);
                    }
                    if (!first) {
                        // what has been accumulated follows, once the products under way
                        // are done: those of the group's chunk before
                        const int gb4 = G::kSplit ? g - 1 : g - 2;
                        ok = wait_warp(bar(G::VRing::free(gb4)), G::VRing::free_parity(gb4), misc);
                    }
                    if (meet(!ok)) {
                        ok = false;
                        break;
                    }
                    pending = (*unset & 1) != 0;
                    wide = (*unset & 2) != 0;
                    if (!first) {
#pragma unroll
                        for (int k = 0; k < R; ++k) l[k] *= alphas[k];
                        umma::fence_after_sync();
#pragma unroll 1
                        for (int c0 = 0; c0 < (G::kLow ? 2 * R : R); c0 += 16) {
                            const uint32_t at = tO + (uint32_t)(c0 < R ? c0 : c0 - R + N);
                            uint32_t o[16];
                            umma::tmem_ld16(at, o);
                            umma::tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * alphas[(c0 & 16) + k]);
                            umma::tmem_st16(at, o);
                        }
                        umma::tmem_wait_st();
                    }
                    load();
                }
                // ---- the weights
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    t[k] = ex2(t[k]);
                    l[k] += t[k];
                }
                if (!G::kSplit) ok = __all_sync(kFull, ok && buffer_free());
                first = false;
                if (ok && there) {
                    const uint32_t pb = sb + (uint32_t)(G::kPOff + (g & 1) * G::kPBuf + key * 128);
#pragma unroll
                    for (int k = 0; k < R; k += 8) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = t[k + 2 * e], b = t[k + 2 * e + 1];
                            if (FP8) {
                                hi[e] = pack_f16x2(a, b);
                                const __half2 h = *reinterpret_cast<const __half2*>(&hi[e]);
                                lo[e] = pack_f16x2(a - __low2float(h), b - __high2float(h));
                            } else {
                                hi[e] = pack_bf16x2(a, b);
                                lo[e] = pack_bf16x2(a - bf16_lo(hi[e]), b - bf16_hi(hi[e]));
                            }
                        }
                        // 16 bytes: eight rows; the low parts N columns on
                        const int ch = (row0 + k) / 8, cl = ch + N / 8;
                        sts128(pb + (uint32_t)((ch >> 3) * kRegion + ((ch ^ key) & 7) * 16),
                               make_uint4(hi[0], hi[1], hi[2], hi[3]));
                        if (G::kLow)
                            sts128(pb + (uint32_t)((cl >> 3) * kRegion + ((cl ^ key) & 7) * 16),
                                   make_uint4(lo[0], lo[1], lo[2], lo[3]));
                    }
                }
                fence_proxy_async_smem();
                umma::fence_before_sync();
                __syncwarp();
                if (ok && lane == 0) {
                    mbar_arrive(bar(G::B_PFULL + (g & 1)));
                    mbar_arrive(bar(G::B_SFREE + (g & 3)));
                }
            }
            // the group's warps go on together, or not at all
            if (meet(!ok)) ok = false;
            if (!ok) break;
            // ---- the segment's result: the sums, and both groups' accumulators
            ok = wait_warp(bar(G::B_OFULL), (uint32_t)(seg & 1), misc);
            umma::fence_after_sync();
            wmax[wq * R + lane] = column_sums(l, lane);
            if (first && wq == 0) ref[lane] = -INFINITY;     // no chunk of this group
            if (meet(!ok)) ok = false;
            if (!ok) break;
            ok = join();
            if (meet(!ok)) ok = false;
            if (!ok) break;
            const bool whole = w.whole();
            const size_t slot = (size_t)cta * 2 + (w.j == 0 ? 1 : 0);
            // a row's factors (of the groups' accumulators, of the result) and its place
            float4* fac = reinterpret_cast<float4*>(gb + G::kFacOff);
            int* rowat = reinterpret_cast<int*>(gb + G::kRowOff);
            if (tid < N) {
                const float* base = reinterpret_cast<const float*>(gb + G::kWmaxOff);
                const float* refs = reinterpret_cast<const float*>(gb + G::kRefOff);
                float s[2] = {0.f, 0.f}, m[2] = {-INFINITY, -INFINITY};
                const int nd = row_node(p, tid);
                // (rows behind the last, and padding nodes, hold what their lanes computed)
                const bool live = tid < rows && !((padw[nd >> 5] >> (nd & 31)) & 1u);
#pragma unroll
                for (int q = 0; q < G::kAccs; ++q) {
                    const int g = G::kSplit ? tid / R : q, r = tid % R;
                    const float* b = base + g * 4 * R + r;
                    m[q] = refs[g * R + r];
                    // (0 for a group without a chunk; NaN among the scores makes it NaN)
                    s[q] = live ? (b[0] + b[R]) + (b[2 * R] + b[3 * R]) : 0.f;
                }
                const float M = fmaxf(m[0], m[1]);
                const float a0 = m[0] == -INFINITY ? 0.f : ex2(m[0] - M);
                const float a1 = m[1] == -INFINITY ? 0.f : ex2(m[1] - M);
                const float L = s[0] * a0 + s[1] * a1;
                float z = 1.f;
                if (whole && L != 0.f) z = p.v_scale / L;
                else if (whole) z = live && sees_any<G::kWords>(w.q, anc + nd * G::kWords) ? __uint_as_float(0x7fffffffu) : 0.f;
                fac[tid] = make_float4(a0, a1, z, L);
                rowat[tid] = whole ? (w.q.t0 + nd) * p.Hq + w.h * p.G + tid - nd * p.G : (int)(slot * N) + tid;
                if (!whole && tid < rows) p.part_ml[slot * N + tid] = make_float2(M, L);
            }
            ok = join();
            if (meet(!ok)) ok = false;
            if (!ok) break;
            // drafted V elements that were zeroed as infinities or NaN
            const volatile uint32_t* badw = reinterpret_cast<const volatile uint32_t*>(gb + G::kBadOff) + buf * G::kPrepWarps * 4;
            bool back = false;
            if (w.drafted(nc - 1))
                for (int q = 0; q < G::kPrepWarps * 4; ++q) back = back || badw[q] != 0u;
            // a thread per dimension (the lower D lanes), half of the rows a group
            if (wq * 32 < D) {
                const int d = key;
#pragma unroll 1
                for (int r0 = grp * (N / 2); r0 < min((grp + 1) * (N / 2), rows); r0 += 16) {
                    float v[16];
                    uint32_t o[16];
                    const uint32_t t0 = lanes + G::kColO + (uint32_t)r0;
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = 0.f;
#pragma unroll
                    for (int q = 0; q < G::kAccs; ++q) {
                        uint32_t low[16];
                        umma::tmem_ld16(t0 + (uint32_t)(q * G::kPW), o);
                        if (G::kLow) umma::tmem_ld16(t0 + (uint32_t)(q * G::kPW + N), low);
                        umma::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float a = q == 0 ? fac[r0 + k].x : fac[r0 + k].y;
                            const float sum = __uint_as_float(o[k]) + (G::kLow ? __uint_as_float(low[k]) : 0.f);
                            if (a != 0.f) v[k] += sum * a;
                        }
                    }
                    if (back) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int nd = row_node(p, r0 + k);
                            if (r0 + k >= rows || ((padw[nd >> 5] >> (nd & 31)) & 1u)) continue;
                            for (int k4 = 0; k4 < G::kWords; ++k4) {
                                uint32_t b = 0u;
                                for (int q = 0; q < G::kPrepWarps; ++q) b |= badw[q * 4 + k4];
                                for (b &= anc[nd * G::kWords + k4]; b != 0u; b &= b - 1u) {
                                    const int pos = w.q.base + 32 * k4 + __ffs(b) - 1;
                                    const int blk = __ldg(p.bt + (size_t)w.s * p.max_blocks + pos / kBlock);
                                    if (blk < 0 || blk >= p.num_blocks) continue;
                                    const size_t at = (((size_t)blk * p.Hkv + w.h) * kBlock + pos % kBlock) * D + d;
                                    if (FP8) {
                                        if ((p.v_cache[at] & 0x7fu) == 0x7fu) v[k] = __uint_as_float(0x7fffffffu);
                                    } else {
                                        const float z = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p.v_cache)[at] << 16);
                                        if (!(fabsf(z) < INFINITY)) v[k] += z;
                                    }
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        if (r0 + k >= rows) break;
                        const float x = v[k] * fac[r0 + k].z;
                        const size_t at = (size_t)rowat[r0 + k] * D + d;
                        if (!whole) p.part_o[at] = x;
                        else if (p.out_f32) static_cast<float*>(p.out)[at] = x;
                        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(x);
                    }
                }
            }
            if (tid == 0 && w.j == 0 && !whole) {
                // the CTA with the first pages says where the partials are
                const int last = (int)(((long long)flat + w.q.nb - 1) / misc[M_Q]);
                p.meta[cta] = make_int4(w.s, w.h, last - cta + 1, rows);
            }
            flat += w.np + kExtraPages;
            g0 += nc;
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(G::B_OFREE + buf));
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == G::kMmaWarp) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, G::kTmemCols);
    }
}

std::mutex g_small_mu;

template <int D, bool FP8, int N>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, cudaStream_t st)
{
    using G = SmallGeo<D, FP8, N>;
    static bool ready[64] = {};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(g_small_mu);
        if (!ready[dev]) {
            if (cudaError_t e = cudaFuncSetAttribute(paged_tree_small_kernel<D, FP8, N>,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem))
                return e;
            ready[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.nctas);
    cfg.blockDim = dim3(G::kThreads);
    cfg.dynamicSmemBytes = G::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_tree_small_kernel<D, FP8, N>, mk, mv, p);
}

}  // namespace

int tree_small_rows(int rows) { return rows <= 32 ? 32 : 64; }

cudaError_t tree_small_launch(const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, int D,
                              bool fp8, int rows, cudaStream_t st)
{
    const bool n32 = tree_small_rows(rows) == 32;
    g_launched.note();
    if (D == 128) {
        if (fp8) return n32 ? launch<128, true, 32>(mk, mv, p, st) : launch<128, true, 64>(mk, mv, p, st);
        return n32 ? launch<128, false, 32>(mk, mv, p, st) : launch<128, false, 64>(mk, mv, p, st);
    }
    if (fp8) return n32 ? launch<64, true, 32>(mk, mv, p, st) : launch<64, true, 64>(mk, mv, p, st);
    return n32 ? launch<64, false, 32>(mk, mv, p, st) : launch<64, false, 64>(mk, mv, p, st);
}

int tree_small_read_error(unsigned* flags, long long* detail) { return g_launched.take_error(g_tree_err, flags, detail); }

}  // namespace pkv
