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
// n * G query rows of a KV head, so up to about 256 rows the time is that of the
// bytes (rows * 4 flop per 2 bytes of a bf16 cache against 1863 TFLOP/s and
// 6.8 TB/s), beyond them that of the exponentials: 16 a clock and SM, one per
// row and key, more than the 2 * D multiply-adds of a row and key take in the
// tensor cores.
//
// How:
//  * The rows of a KV head's nodes (row r = node * G + head) fill tiles of 128
//    rows, one MMA's M.  A CTA works on one tile (TILES == 1) or two (TILES ==
//    2, when a tree may have more than 128 rows); more tiles than that are
//    served by as many teams of CTAs, which cut the same keys the same way, so
//    that the repeated reads of a tile of keys come at about the same time and
//    hit L2.
//  * One persistent CTA per SM takes an equal contiguous range of the flat
//    (sequence, KV head, page) list and consumes it in chunks of up to 8 pages
//    (128 keys).  Warp 8 streams K and V of a chunk through a ring with TMA.
//  * Two streams work side by side, each with its own MMA warp (9, 10), four
//    softmax warps (0-3, 4-7; one row a thread) and half of tensor memory: the
//    scores S (128 columns), overwritten in place by the weights P, and the
//    accumulator O.  With TILES == 2 a stream has its own row tile and both
//    consume every chunk; with TILES == 1 they take the chunks in turn and
//    their two results are joined at the end of the range.  So one stream's
//    matrix products run under the other's exponentials.
//  * S = Q K^T with K as it lies in the ring; P is written as bf16 high and low
//    parts (a bf16 cache; so weights keep 16 bits and an output is not
//    further off than its own rounding) or as f16 (an E4M3 cache, whose tiles
//    warps 11-14 widen to f16, which holds every code exactly); O += P V.
//  * Only the chunks that reach the drafted positions need masks; there warp 11
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
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "cache_map.h"
#include "device_common.cuh"
#include "internal.h"
#include "paged_kv.h"
#include "tree_common.cuh"
#include "umma.cuh"

namespace pkv {

__device__ DevErr g_tree_err;

namespace {

constexpr int kTile = 128;                      // rows of a tile: M of every MMA
constexpr int kPages = 8;                       // pages of a chunk
constexpr int kKeys = kPages * kBlock;
constexpr int kN = KV_TREE_MAX_NODES;
constexpr uint32_t kTmemCols = 512;             // S0, S1, O0, O1: 128 columns each
constexpr long long kWaitLimit = 1LL << 31;     // ~1 s of SM clocks
constexpr float kMaxLag = 8.f;                  // the reference maximum may lag by 2^8
// f16 weights carry a factor of 2^7: at most 2^15 with the lag, and what f16
// rounds to zero is below 2^-31 of the largest weight
constexpr float kBiasF16 = 7.f;

// Columns of O joined at a time, and the floats between two rows of them.
constexpr int kStageCols = 16, kStageRow = 17;

// Few rows leave most of a tile's 128 lanes empty.  They are then repeated: R
// copies of up to 128 / R rows, copy i (a quarter or a half of the lanes, the
// warps that own them) with the weights of the i-th share of each chunk's keys
// and zeros for the rest, so that the exponentials are spread over all warps.
__host__ __device__ constexpr int row_copies(int rows)
{
    return rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
}

// A stream's chunks: every second one, or all.
constexpr int chunk_step(int tiles) { return tiles == 1 ? 2 : 1; }

template <int D, bool FP8, int TILES>
struct Geo {
    static constexpr int kPrepWarp = 11;                     // first of the prep / widening warps
    static constexpr int kPrepWarps = FP8 ? 4 : 1;
    static constexpr int kWarps = kPrepWarp + kPrepWarps;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kBoxes = D / 64;                    // 128-byte column groups of a row
    static constexpr int kRegion = kKeys * 128;              // one column group of a chunk
    static constexpr int kSlot = kBoxes * kRegion;           // K or V of a chunk, 2 bytes each
    static constexpr int kQTile = kBoxes * kTile * 128;
    static constexpr int kPageBytes = kBlock * D * (FP8 ? 1 : 2);
    static constexpr int kRawSlot = kPages * kBlock * D;     // E4M3 codes of K or V of a chunk
    // slots the MMAs read (filled by TMA, or by the widening warps), and the
    // ring of codes in front of them
    static constexpr int kSlots = FP8 ? (D == 128 ? 3 : 6)
                                      : (TILES == 1 ? 5 : 4) * (D == 128 ? 1 : 2);
    static constexpr int kRawSlots = !FP8 ? 0 : (TILES == 1 ? 4 : 3) * (D == 128 ? 1 : 2);
    static constexpr int kLoadSlots = FP8 ? kRawSlots : kSlots;
    static constexpr int kQOff = 0;
    static constexpr int kSlotOff = kQOff + TILES * kQTile;
    static constexpr int kRawOff = kSlotOff + kSlots * kSlot;
    static constexpr int kBarOff = kRawOff + kRawSlots * kRawSlot;
    // barriers
    static constexpr int B_FULL = 0;                         // + load slot: the copies have landed
    static constexpr int B_EMPTY = B_FULL + kLoadSlots;      // + load slot: it may be refilled
    static constexpr int B_WIDE = B_EMPTY + kLoadSlots;      // + slot: widened (FP8)
    static constexpr int B_WFREE = B_WIDE + (FP8 ? kSlots : 0);  // + slot: the MMAs have read it
    static constexpr int B_FIX = B_WFREE + (FP8 ? kSlots : 0);   // + slot: V rows fixed (bf16)
    static constexpr int B_QFULL = B_FIX + (FP8 ? 0 : kSlots);   // Q and the tree of a segment
    static constexpr int B_QFREE = B_QFULL + 1;              // its last scores are computed
    static constexpr int B_SFULL = B_QFREE + 1;              // + stream
    static constexpr int B_PFULL = B_SFULL + 2;              // + stream
    static constexpr int B_PVDONE = B_PFULL + 2;             // + stream
    static constexpr int B_OFULL = B_PVDONE + 2;             // both accumulators are complete
    static constexpr int B_OFREE = B_OFULL + 1;              // + segment & 1: they have been read
    static constexpr int B_ML = B_OFREE + 2;                 // partial (max, sum)s are written
    static constexpr int B_STAGE = B_ML + 1;                 // staged partials are written / read
    static constexpr int B_END = B_STAGE + 1;                // + stream: all its MMAs are done
    static constexpr int B_STALL = B_END + 2;                // nothing arrives (the test hook)
    static constexpr int kNumBars = B_STALL + 1;
    static constexpr int kMiscOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kAncOff = kMiscOff + 64;            // [2][kN][4] words
    static constexpr int kPtrOff = kAncOff + 2 * kN * 16;    // [kN] bytes used by pointer jumping
    static constexpr int kPadOff = kPtrOff + kN * 4;         // [2][4] words
    static constexpr int kBadOff = kPadOff + 32;             // [2][kPrepWarps][4] words
    // the warps whose partial results of a row are joined in the CTA: those of
    // both streams (TILES == 1) or of one
    static constexpr int kJoinWarps = TILES == 1 ? 8 : 4;
    static constexpr int kMlOff = kBadOff + 2 * kPrepWarps * 16;  // [kJoinWarps][32] float2
    static constexpr int kStageOff = kMlOff + kJoinWarps * 32 * 8;  // [kJoinWarps][32][kStageRow]
    static constexpr int kQfacOff = kStageOff + kJoinWarps * 32 * kStageRow * 4;
    static constexpr int kEnd = kQfacOff + (FP8 ? 2 * TILES * kTile * 4 : 0);
    static constexpr int kSmem = kEnd + 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
};

// misc words: tensor-memory base; abort; the range: first unit, units, units per
// CTA, first sequence, KV head and page; halves handed to the ring the MMAs read
enum Misc { M_TMEM = 0, M_ABORT, M_B0, M_CNT, M_Q, M_S0, M_H0, M_J0, M_ISSUED };

struct TreeParams {
    const uint16_t* q;          // bf16 [total][Hq][D]
    void* out;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const int32_t* bt;
    const int32_t* ctx;
    const int32_t* starts;
    const int32_t* parents;
    float* part_o;              // [grid][2][TILES * 128][D]
    float2* part_ml;            // [grid][2][TILES * 128]: (max in log2 units, sum)
    int4* meta;                 // [grid]: (sequence, KV head, partials, rows)
    int B, total, max_nodes, Hq, Hkv, G, max_blocks, num_blocks;
    uint32_t g_magic;           // ceil(2^32 / G), 0 for G == 1
    int nctas;                  // CTAs of a team
    int teams;
    int min_q;                  // least pages of a CTA's range
    float sl2, v_scale;
    int out_f32;
    long long test_stall;
};

__device__ __forceinline__ void pdl_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void pdl_launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
}

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
            raise_flag(&g_tree_err, KV_DEVERR_PIPELINE_TIMEOUT, blockIdx.x);
            return false;
        }
    }
}

// Wait until half x is on its way into its slot.  A role that does not follow
// every half of a ring (a stream that takes every second chunk, the warp that
// fixes V rows) does this before it waits for the half's barrier: the slot's
// previous phase is then known to be over, and the phase's parity to be that of
// half x.
__device__ __forceinline__ bool wait_issued(int x, volatile int* misc)
{
    if (misc[M_ISSUED] > x) return true;
    const long long t0 = clock64();
    while (misc[M_ISSUED] <= x) {
        if (misc[M_ABORT]) return false;
        if (clock64() - t0 > kWaitLimit) {
            misc[M_ABORT] = 1;
            raise_flag(&g_tree_err, KV_DEVERR_PIPELINE_TIMEOUT, blockIdx.x);
            return false;
        }
    }
    return true;
}

// The same for a whole warp.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* misc)
{
    return __all_sync(kFull, wait_bar(bar, parity, misc));
}

__device__ __forceinline__ long long warp_sum_ll(long long v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// One sequence as a team sees it.
struct SeqInfo {
    int t0, n, L, base, nb;     // nb: pages, 0 when the team has no rows here
};

template <int TILES>
__device__ __forceinline__ SeqInfo seq_info(const TreeParams& p, int s, int team, bool flag)
{
    SeqInfo q;
    int bad = 0;
    if (!tree_span(p.starts, s, p.total, p.max_nodes, q.t0, q.n, bad) && flag)
        raise_flag(&g_tree_err, KV_DEVERR_BAD_TREE, bad);
    int L = __ldg(p.ctx + s);
    const int cap = p.max_blocks * kBlock;
    if (L < 0 || L > cap) {
        if (flag) raise_flag(&g_tree_err, KV_DEVERR_CONTEXT_TOO_LONG, L);
        L = L < 0 ? 0 : cap;
    }
    if (flag && L > 0 && L < q.n) raise_flag(&g_tree_err, KV_DEVERR_BAD_TREE, L);
    q.L = L;
    q.base = L > q.n ? L - q.n : 0;
    q.nb = q.n * p.G > team * TILES * kTile ? (L + kBlock - 1) / kBlock : 0;
    return q;
}

// Node (within the sequence) of row r of a KV head's rows.
__device__ __forceinline__ int row_node(const TreeParams& p, int r)
{
    return p.g_magic ? (int)__umulhi((uint32_t)r, p.g_magic) : r;
}

// The segments of a CTA's range: the pages [j, j + np) of one (sequence, KV
// head) each.  Every role walks the same list.
template <int TILES>
struct Walk {
    int s, h, j, rem, seg, np;
    SeqInfo q;
    __device__ __forceinline__ Walk(const TreeParams& p, const volatile int* misc, int team)
    {
        s = misc[M_S0];
        h = misc[M_H0];
        j = misc[M_J0];
        rem = misc[M_CNT];
        seg = 0;
        np = 0;
        if (rem > 0) {
            q = seq_info<TILES>(p, s, team, false);
            np = min(q.nb - j, rem);
        }
    }
    __device__ __forceinline__ bool more() const { return rem > 0; }
    __device__ __forceinline__ int chunks() const { return (np + kPages - 1) / kPages; }
    __device__ __forceinline__ int chunk_pages(int c) const { return min(kPages, np - c * kPages); }
    // does chunk c reach the drafted positions?
    __device__ __forceinline__ bool drafted(int c) const
    {
        return (j + c * kPages + chunk_pages(c)) * kBlock > q.base;
    }
    __device__ __forceinline__ void next(const TreeParams& p, int team)
    {
        rem -= np;
        ++seg;
        if (rem <= 0) return;
        j = 0;
        if (++h == p.Hkv) {
            h = 0;
            do {
                if (++s >= p.B) {
                    rem = 0;
                    return;
                }
                q = seq_info<TILES>(p, s, team, false);
            } while (q.nb == 0);
        }
        np = min(q.nb, rem);
    }
};

// Byte offset of 16-byte chunk c of row r in a [128 rows x 128 B] region
// (128-byte swizzle).
__device__ __forceinline__ uint32_t region_off(int r, int c)
{
    return (uint32_t)(r * 128) + (uint32_t)(((c ^ (r & 7)) & 7) * 16);
}

// Two E4M3 codes (the low half of x) as two f16: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(x));
    return r;
}

// Zero the infinities and NaN (bf16), or NaN (E4M3), of four elements' words;
// true if there were any.
template <bool FP8>
__device__ __forceinline__ bool drop_non_finite(uint32_t (&x)[4])
{
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t m = FP8 ? __vcmpeq4(x[k] & 0x7f7f7f7fu, 0x7f7f7f7fu)
                               : __vcmpeq2(x[k] & 0x7f807f80u, 0x7f807f80u);
        x[k] &= ~m;
        any |= m;
    }
    return any != 0;
}

template <int D, bool FP8, int TILES>
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
    volatile int* misc = reinterpret_cast<volatile int*>(gb + G::kMiscOff);
    auto bar = [&](int i) -> uint32_t { return sb + (uint32_t)(G::kBarOff + 8 * i); };
    uint32_t* anc = reinterpret_cast<uint32_t*>(gb + G::kAncOff);
    volatile uint32_t* padw = reinterpret_cast<volatile uint32_t*>(gb + G::kPadOff);
    volatile uint32_t* badw = reinterpret_cast<volatile uint32_t*>(gb + G::kBadOff);

    if (tid == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        constexpr int kReaders = TILES;          // MMA warps that read every slot
        for (int i = 0; i < G::kLoadSlots; ++i) {
            mbar_init(bar(G::B_FULL + i), 1);
            mbar_init(bar(G::B_EMPTY + i), FP8 ? G::kPrepWarps : kReaders);
        }
        if (FP8)
            for (int i = 0; i < G::kSlots; ++i) {
                mbar_init(bar(G::B_WIDE + i), G::kPrepWarps);
                mbar_init(bar(G::B_WFREE + i), kReaders);
            }
        else
            for (int i = 0; i < G::kSlots; ++i) mbar_init(bar(G::B_FIX + i), 1);
        mbar_init(bar(G::B_QFULL), G::kPrepWarps);
        mbar_init(bar(G::B_QFREE), 2);
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar(G::B_SFULL + w), 1);
            mbar_init(bar(G::B_PFULL + w), 4);
            mbar_init(bar(G::B_PVDONE + w), 1);
            mbar_init(bar(G::B_OFREE + w), 8);
            mbar_init(bar(G::B_END + w), 1);
        }
        mbar_init(bar(G::B_OFULL), 2);
        mbar_init(bar(G::B_ML), G::kJoinWarps);
        mbar_init(bar(G::B_STAGE), G::kJoinWarps);
        mbar_init(bar(G::B_STALL), 1);
        misc[M_ABORT] = 0;
        misc[M_ISSUED] = 0;
        fence_mbar_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    if (warp == 9) {
        umma::tmem_alloc(sb + G::kMiscOff + 4 * M_TMEM, kTmemCols);
        umma::tmem_relinquish();
    }
    if (warp == 8) {
        // this CTA's range of the team's flat (sequence, KV head, page) list
        const bool flag = blockIdx.x == 0;
        long long total = 0;
        for (int b = 0; b < p.B; b += 32) {
            int nb = 0;
            if (b + lane < p.B) nb = seq_info<TILES>(p, b + lane, team, flag).nb;
            total += warp_sum_ll(nb);
        }
        total *= p.Hkv;
        long long q = (total + p.nctas - 1) / p.nctas;
        if (q < p.min_q) q = p.min_q;
        const long long b0 = (long long)cta * q;
        long long cnt = total - b0;
        if (cnt > q) cnt = q;
        if (cnt < 0) cnt = 0;
        int s0 = 0, h0 = 0, j0 = 0;
        if (cnt > 0) {
            long long excl = 0;
            bool found = false;
            for (int b = 0; b < p.B && !found; b += 32) {
                int nb = 0;
                if (b + lane < p.B) nb = seq_info<TILES>(p, b + lane, team, false).nb;
                const long long v = (long long)nb * p.Hkv;
                long long inc = v;
                for (int o = 1; o < 32; o <<= 1) {
                    const long long t = __shfl_up_sync(kFull, inc, o);
                    if (lane >= o) inc += t;
                }
                inc += excl;
                const unsigned m = __ballot_sync(kFull, inc > b0);
                if (m) {
                    const int src = __ffs(m) - 1;
                    const long long ex = __shfl_sync(kFull, inc - v, src);
                    const int nbs = __shfl_sync(kFull, nb, src);
                    s0 = b + src;
                    const long long off = b0 - ex;
                    h0 = (int)(off / nbs);
                    j0 = (int)(off - (long long)h0 * nbs);
                    found = true;
                }
                excl = __shfl_sync(kFull, inc, 31);
            }
            if (!found) cnt = 0;
        }
        if (lane == 0) {
            misc[M_B0] = (int)b0;
            misc[M_CNT] = (int)cnt;
            misc[M_Q] = (int)q;
            misc[M_S0] = s0;
            misc[M_H0] = h0;
            misc[M_J0] = j0;
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = (uint32_t)misc[M_TMEM];

    if (warp == 8) {
        // ------------------------------------------------------------- copies
        const uint64_t pol = l2_evict_first_policy();
        int x = 0;                               // halves (K or V of a chunk) issued
        bool ok = true;
        for (Walk<TILES> w(p, misc, team); ok && w.more(); w.next(p, team)) {
            const int32_t* row = p.bt + (size_t)w.s * p.max_blocks + w.j;
            int ids = lane < w.np ? __ldg(row + lane) : -1;       // pages 0..31 of the segment
            int ahead = 32 + lane < w.np ? __ldg(row + 32 + lane) : -1;
            const int nc = w.chunks();
            for (int c = 0; ok && c < nc; ++c) {
                if (c > 0 && (c & 3) == 0) {
                    ids = ahead;
                    const int at = (c + 4) * kPages + lane;
                    ahead = at < w.np ? __ldg(row + at) : -1;
                }
                const int np = w.chunk_pages(c);
                const int id = __shfl_sync(kFull, ids, (c & 3) * kPages + lane / G::kBoxes % kPages);
                const int box = FP8 ? 0 : lane % G::kBoxes;
                const int page = FP8 ? lane : lane / G::kBoxes;
                const int my = FP8 ? __shfl_sync(kFull, ids, (c & 3) * kPages + (lane & 7)) : id;
                const bool mine = page < np;
                const bool valid = mine && my >= 0 && my < p.num_blocks;
                if (mine && !valid && box == 0) raise_flag(&g_tree_err, KV_DEVERR_BLOCK_OUT_OF_RANGE, my);
                const int nvalid = __popc(__ballot_sync(kFull, valid && box == 0));
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++x) {
                    const int slot = x % G::kLoadSlots, round = x / G::kLoadSlots;
                    if (round > 0) ok = wait_warp(bar(G::B_EMPTY + slot), (uint32_t)((round - 1) & 1), misc);
                    if (!ok) break;
                    const uint32_t fb = bar(G::B_FULL + slot);
                    if (lane == 0) {
                        if (nvalid > 0) mbar_arrive_expect_tx(fb, (uint32_t)(nvalid * G::kPageBytes));
                        else mbar_arrive(fb);
                    }
                    __syncwarp();
                    if (valid) {
                        const uint32_t dst =
                            FP8 ? sb + (uint32_t)(G::kRawOff + slot * G::kRawSlot + page * G::kPageBytes)
                                : sb + (uint32_t)(G::kSlotOff + slot * G::kSlot + box * G::kRegion +
                                                  page * kBlock * 128);
                        const void* tm = kv == 0 ? &tm_k : &tm_v;
                        const int z = my * p.Hkv + w.h;
                        if (p.teams == 1)        // read once: first out of L2
                            tma_load_3d_hint(dst, tm, box * 64, 0, z, fb, pol);
                        else
                            tma_load_3d(dst, tm, box * 64, 0, z, fb);
                    }
                    if (!FP8 && lane == 0) misc[M_ISSUED] = x + 1;
                }
            }
        }
        // every issued copy lands before the CTA can end
        if (lane == 0)
            for (int i = x > G::kLoadSlots ? x - G::kLoadSlots : 0; i < x; ++i)
                mbar_wait_bounded(bar(G::B_FULL + i % G::kLoadSlots),
                                  (uint32_t)((i / G::kLoadSlots) & 1), kWaitLimit);
        __syncwarp();
    } else if (warp == 9 || warp == 10) {
        // --------------------------------------------------------------- MMAs
        if (lane == 0) {
            const int st = warp - 9;
            const uint32_t tS = tmem + (uint32_t)(128 * st), tO = tmem + 256u + (uint32_t)(128 * st);
            const uint64_t qdesc =
                umma::smem_desc_sw128(sb + G::kQOff + (TILES == 2 ? st * G::kQTile : 0), 16, 1024);
            const uint64_t sdesc = umma::smem_desc_sw128(sb + G::kSlotOff, 16, 1024);
            const uint64_t vdesc = umma::smem_desc_sw128(sb + G::kSlotOff, G::kRegion, 1024);
            constexpr uint32_t idesc_pv = FP8 ? umma::idesc_f16_f32(kTile, D, false, true)
                                              : umma::idesc_bf16_f32(kTile, D, false, true);
            const int full0 = FP8 ? G::B_WIDE : G::B_FULL, free0 = FP8 ? G::B_WFREE : G::B_EMPTY;
            uint32_t fix_parity = 0;             // bit slot: parity of its next fix
            int x0 = 0, pc = 0;                  // first half of the segment; chunks of the stream
            bool ok = true;
            if (p.test_stall > 0 && misc[M_CNT] > 0 &&
                !mbar_wait_bounded(bar(G::B_STALL), 0u, p.test_stall)) {
                misc[M_ABORT] = 1;
                raise_flag(&g_tree_err, KV_DEVERR_PIPELINE_TIMEOUT, blockIdx.x);
                ok = false;
            }
            for (Walk<TILES> w(p, misc, team); ok && w.more(); w.next(p, team)) {
                const int nc = w.chunks(), seg = w.seg;
                ok = wait_bar(bar(G::B_QFULL), (uint32_t)(seg & 1), misc);
                if (!ok) break;
                // a second row tile without rows takes no part, but frees the slots
                const bool idle = TILES == 2 && st == 1 &&
                                  w.q.n * p.G - team * TILES * kTile <= kTile;
                bool first = true;
                for (int c = 0; ok && c < nc; ++c) {
                    const int kx = x0 + 2 * c, vx = kx + 1;
                    const int ks = kx % G::kSlots, vs = vx % G::kSlots;
                    const uint32_t kp = (uint32_t)((kx / G::kSlots) & 1);
                    const uint32_t vp = (uint32_t)((vx / G::kSlots) & 1);
                    const bool fix = !FP8 && w.drafted(c);
                    const uint32_t fixp = (fix_parity >> vs) & 1u;
                    if (fix) fix_parity ^= 1u << vs;
                    if (TILES == 1 && (c & 1) != st) continue;
                    ok = wait_issued(kx, misc) && wait_bar(bar(full0 + ks), kp, misc);
                    if (!ok) break;
                    if (idle) {
                        mbar_arrive(bar(free0 + ks));
                        ok = wait_issued(vx, misc) && wait_bar(bar(full0 + vs), vp, misc);
                        if (ok) mbar_arrive(bar(free0 + vs));
                        continue;
                    }
                    const int np = w.chunk_pages(c);
                    // S = Q K^T; the stream's previous P.V products, which read what S
                    // overwrites, are done (PVDONE below)
                    umma::fence_after_sync();
                    {
                        const uint64_t kd = sdesc + (uint64_t)((ks * G::kSlot) >> 4);
                        const uint32_t idesc =
                            FP8 ? umma::idesc_f16_f32(kTile, kBlock * np, false, false)
                                : umma::idesc_bf16_f32(kTile, kBlock * np, false, false);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t a = qdesc + (uint64_t)(((kk >> 2) * kTile * 128 + (kk & 3) * 32) >> 4);
                            const uint64_t b = kd + (uint64_t)(((kk >> 2) * G::kRegion + (kk & 3) * 32) >> 4);
                            umma::mma_bf16_ss(tS, a, b, idesc, kk > 0);
                        }
                    }
                    umma::commit(bar(G::B_SFULL + st));
                    umma::commit(bar(free0 + ks));
                    if (c + chunk_step(TILES) >= nc) umma::commit(bar(G::B_QFREE));
                    ok = wait_bar(bar(G::B_PFULL + st), (uint32_t)(pc & 1), misc);
                    if (!ok) break;
                    ok = wait_issued(vx, misc) && wait_bar(bar(full0 + vs), vp, misc);
                    if (ok && fix) ok = wait_bar(bar(G::B_FIX + vs), fixp, misc);
                    if (ok && first && seg > 0)
                        ok = wait_bar(bar(G::B_OFREE + ((seg - 1) & 1)), (uint32_t)(((seg - 1) >> 1) & 1), misc);
                    if (!ok) break;
                    umma::fence_after_sync();
                    {
                        const uint64_t vd = vdesc + (uint64_t)((vs * G::kSlot) >> 4);
                        for (int kk = 0; kk < np; ++kk) {
                            // the weights of keys 16 kk .. 16 kk + 15: 8 columns of the
                            // 32 that held the scores of 32 keys; their low parts 16 on
                            const uint32_t a = tS + (uint32_t)(32 * (kk >> 1) + 8 * (kk & 1));
                            const uint64_t b = vd + (uint64_t)((kk * kBlock * 128) >> 4);
                            umma::mma_bf16_ts(tO, a, b, idesc_pv, !(first && kk == 0));
                            if (!FP8) umma::mma_bf16_ts(tO, a + 16u, b, idesc_pv, true);
                        }
                    }
                    umma::commit(bar(free0 + vs));
                    umma::commit(bar(G::B_PVDONE + st));
                    first = false;
                    ok = wait_bar(bar(G::B_PVDONE + st), (uint32_t)(pc & 1), misc);
                    ++pc;
                }
                if (!ok) break;
                x0 += 2 * nc;
                // a stream without a chunk arrives for both; not before the other
                // stream has for the segment before
                if (first) {
                    mbar_arrive(bar(G::B_QFREE));
                    if (seg > 0) ok = wait_bar(bar(G::B_OFULL), (uint32_t)((seg - 1) & 1), misc);
                    if (!ok) break;
                }
                umma::fence_after_sync();
                umma::fence_before_sync();
                mbar_arrive(bar(G::B_OFULL));
            }
            // every MMA issued by this thread is complete before the CTA ends
            umma::commit(bar(G::B_END + st));
            mbar_wait_bounded(bar(G::B_END + st), 0u, kWaitLimit);
        }
        __syncwarp();
    } else if (warp >= G::kPrepWarp) {
        // ------------------------- queries, trees, V rows, and widening (E4M3)
        const int pw = warp - G::kPrepWarp;
        int x0 = 0;
        bool ok = true;
        for (Walk<TILES> w(p, misc, team); ok && w.more(); w.next(p, team)) {
            const int seg = w.seg, buf = seg & 1, nc = w.chunks(), n = w.q.n;
            // the segment's entry of the tree tables was last read two segments ago
            if (seg >= 2) ok = wait_warp(bar(G::B_OFREE + buf), (uint32_t)(((seg - 2) >> 1) & 1), misc);
            if (ok && seg >= 1) ok = wait_warp(bar(G::B_QFREE), (uint32_t)((seg - 1) & 1), misc);
            if (!ok) break;
            if (lane < 4) badw[(buf * G::kPrepWarps + pw) * 4 + lane] = 0u;
            // ---- the query rows of the team's tiles
            const int r0 = team * TILES * kTile;
            const int rows = min(n * p.G - r0, TILES * kTile);
            const int copies = row_copies(n * p.G - r0), stride = kTile / copies;
            constexpr int C = D / 8;             // 16-byte chunks (8 elements) of a row
            constexpr int RI = 32 / C;           // rows of a warp's instruction
            const int c = lane % C;
            for (int rb = pw * RI; rb < rows; rb += G::kPrepWarps * RI) {
                const int r = rb + lane / C;
                const int rc = min(r, rows - 1);
                const int node = row_node(p, r0 + rc), g = r0 + rc - node * p.G;
                const uint16_t* src =
                    p.q + ((size_t)(w.q.t0 + node) * p.Hq + (size_t)w.h * p.G + g) * D + 8 * c;
                const uint32_t dst = sb + (uint32_t)(G::kQOff + (rc >> 7) * G::kQTile + (c >> 3) * kTile * 128) +
                                     region_off(rc & 127, c & 7);
                // (a copy's rows are a multiple of 8 on: the same place in the swizzle)
                if (!FP8) {
                    if (r < rows)
                        for (int k = 0; k < copies; ++k) cp_async16(dst + (uint32_t)(k * stride * 128), src);
                } else {
                    // f16 overflows above 65504: a row whose largest |element| is 2^15
                    // or more is divided by a power of two that brings it below (exact
                    // but for elements below 2^-39 of the largest), which the scores
                    // are multiplied by again
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
                    const uint32_t q4[4] = {v.x, v.y, v.z, v.w};
                    uint32_t big = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        big = max(big, max(q4[k] & 0x7fffu, (q4[k] >> 16) & 0x7fffu));
#pragma unroll
                    for (int o = C / 2; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(kFull, big, o));
                    const int e = (int)(big >> 7) - (127 + 14);
                    const float down = e > 0 ? __uint_as_float((uint32_t)(127 - min(e, 126)) << 23) : 1.f;
                    const float up = e > 0 ? __uint_as_float((uint32_t)(127 + min(e, 126)) << 23) : 1.f;
                    uint32_t h4[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h4[k] = pack_f16x2(bf16_lo(q4[k]) * down, bf16_hi(q4[k]) * down);
                    if (r < rows) {
                        for (int k = 0; k < copies; ++k)
                            sts128(dst + (uint32_t)(k * stride * 128), make_uint4(h4[0], h4[1], h4[2], h4[3]));
                        if (c == 0)
                            reinterpret_cast<volatile float*>(gb + G::kQfacOff)[buf * TILES * kTile + r] = up;
                    }
                }
            }
            // ---- the nodes each node sees, by doubling along the parents
            if (pw == 0) {
                volatile int* ptr = reinterpret_cast<volatile int*>(gb + G::kPtrOff);
                volatile uint32_t* am = anc + buf * kN * 4;
                int up[kN / 32];
                uint32_t m[kN / 32][4];
#pragma unroll
                for (int k = 0; k < kN / 32; ++k) {
                    const int i = 32 * k + lane;
                    int par = -1;
                    if (i < n)
                        par = tree_parent(p.parents, w.q.t0, i,
                                          w.h == 0 && w.j == 0 ? &g_tree_err : nullptr);
                    const bool pad = i < n && par == KV_TREE_PAD;
                    const unsigned pads = __ballot_sync(kFull, pad);
                    if (lane == 0) padw[buf * 4 + k] = pads;
                    up[k] = i < n && !pad ? par : -1;
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        m[k][v] = v == k && i < n && !pad ? 1u << lane : 0u;
                }
                for (int reach = 1; reach < n; reach *= 2) {
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < kN / 32; ++k) {
                        const int i = 32 * k + lane;
                        ptr[i] = up[k];
#pragma unroll
                        for (int v = 0; v < 4; ++v) am[4 * i + v] = m[k][v];
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < kN / 32; ++k) {
                        if (up[k] >= 0) {
                            const int a = up[k];
#pragma unroll
                            for (int v = 0; v < 4; ++v) m[k][v] |= am[4 * a + v];
                            up[k] = ptr[a];
                        }
                    }
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < kN / 32; ++k)
#pragma unroll
                    for (int v = 0; v < 4; ++v) am[4 * (32 * k + lane) + v] = m[k][v];
            }
            if (!FP8) cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(G::B_QFULL));

            if constexpr (!FP8) {
                // ---- V rows of the chunks that reach the drafted positions
                for (int ch = 0; ok && ch < nc; ++ch) {
                    if (!w.drafted(ch)) continue;
                    const int vx = x0 + 2 * ch + 1, slot = vx % G::kSlots;
                    ok = __all_sync(kFull, wait_issued(vx, misc)) &&
                         wait_warp(bar(G::B_FULL + slot), (uint32_t)((vx / G::kSlots) & 1), misc);
                    if (!ok) break;
                    const uint32_t vb = sb + (uint32_t)(G::kSlotOff + slot * G::kSlot);
                    const int p0 = (w.j + ch * kPages) * kBlock;
                    const int lo = max(0, w.q.base - p0), hi = w.chunk_pages(ch) * kBlock;
                    for (int rb = lo; rb < hi; rb += RI) {
                        const int r = rb + lane / C;
                        const uint32_t at = vb + (uint32_t)((c >> 3) * G::kRegion) + region_off(r & 127, c & 7);
                        const bool in = r < hi, tail = p0 + r >= w.q.L;
                        if (!in) continue;
                        uint32_t v[4] = {0u, 0u, 0u, 0u};
                        bool bad = false;
                        if (!tail) {
                            lds128(v, at);
                            bad = drop_non_finite<false>(v);
                        }
                        if (tail || bad) sts128(at, make_uint4(v[0], v[1], v[2], v[3]));
                        if (bad) {
                            const int a = p0 + r - w.q.base;
                            atomicOr(const_cast<uint32_t*>(&badw[(buf * G::kPrepWarps + pw) * 4 + (a >> 5)]),
                                     1u << (a & 31));
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(G::B_FIX + slot));
                }
            } else {
                // ---- widen K and V of every chunk: 16 codes a thread and step
                constexpr int CR = D / 16;           // 16-code pieces of a row
                constexpr int RS = 128 / CR;         // rows of the four warps' step
                const int t = pw * 32 + lane;
                const int cc = t % CR;
                for (int ch = 0; ok && ch < nc; ++ch) {
                    const int keys = w.chunk_pages(ch) * kBlock;
                    const int p0 = (w.j + ch * kPages) * kBlock;
                    const bool drafted = w.drafted(ch);
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv) {
                        const int hx = x0 + 2 * ch + kv;
                        const int rs = hx % G::kRawSlots, slot = hx % G::kSlots;
                        ok = wait_warp(bar(G::B_FULL + rs), (uint32_t)((hx / G::kRawSlots) & 1), misc);
                        if (ok && hx >= G::kSlots)
                            ok = wait_warp(bar(G::B_WFREE + slot), (uint32_t)((hx / G::kSlots - 1) & 1), misc);
                        if (!ok) break;
                        if (pw == 0 && lane == 0) misc[M_ISSUED] = hx + 1;
                        const uint32_t raw = sb + (uint32_t)(G::kRawOff + rs * G::kRawSlot);
                        const uint32_t dst = sb + (uint32_t)(G::kSlotOff + slot * G::kSlot);
                        // the copy's swizzle: 16-byte pieces XOR bits 7 and up
                        auto load = [&](int r, uint32_t (&v)[4]) {
                            const uint32_t a = (uint32_t)(r * D + cc * 16);
                            lds128(v, raw + (a ^ (((a >> 7) & (D == 128 ? 7u : 3u)) << 4)));
                        };
                        // (the pieces of the second column group go in the other order:
                        // the eight lanes of a row then write to all banks at once)
                        auto store = [&](int r, const uint32_t (&v)[4]) {
                            const uint32_t d0 = dst + (uint32_t)((cc >> 2) * G::kRegion);
                            uint4 o[2];
                            o[0] = make_uint4(e4m3x2_to_f16x2(v[0]), e4m3x2_to_f16x2(v[0] >> 16),
                                              e4m3x2_to_f16x2(v[1]), e4m3x2_to_f16x2(v[1] >> 16));
                            o[1] = make_uint4(e4m3x2_to_f16x2(v[2]), e4m3x2_to_f16x2(v[2] >> 16),
                                              e4m3x2_to_f16x2(v[3]), e4m3x2_to_f16x2(v[3] >> 16));
                            const int second = (cc >> 2) & 1;
                            sts128(d0 + region_off(r, (2 * cc + second) & 7), second ? o[1] : o[0]);
                            sts128(d0 + region_off(r, (2 * cc + 1 - second) & 7), second ? o[0] : o[1]);
                        };
                        if (keys == kKeys && !(kv == 1 && drafted)) {
                            constexpr int kStep = 4;         // loads in flight
#pragma unroll
                            for (int rb = 0; rb < kKeys; rb += kStep * RS) {
                                uint32_t v[kStep][4];
#pragma unroll
                                for (int k = 0; k < kStep; ++k) load(rb + k * RS + t / CR, v[k]);
#pragma unroll
                                for (int k = 0; k < kStep; ++k) store(rb + k * RS + t / CR, v[k]);
                            }
                        } else {
                            for (int rb = 0; rb < keys; rb += RS) {
                                const int r = rb + t / CR, pos = p0 + r;
                                if (r >= keys) continue;
                                uint32_t v[4];
                                load(r, v);
                                if (kv == 1 && pos >= w.q.L) {
                                    v[0] = v[1] = v[2] = v[3] = 0u;
                                } else if (kv == 1 && pos >= w.q.base && drop_non_finite<true>(v)) {
                                    const int an = pos - w.q.base;
                                    atomicOr(const_cast<uint32_t*>(&badw[(buf * G::kPrepWarps + pw) * 4 + (an >> 5)]),
                                             1u << (an & 31));
                                }
                                store(r, v);
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(bar(G::B_EMPTY + rs));
                            mbar_arrive(bar(G::B_WIDE + slot));
                        }
                    }
                }
            }
            x0 += 2 * nc;
        }
        if (!FP8) cp_async_wait_all();
    } else {
        // ------------------------------------------------- softmax and output
        const int st = warp >> 2;                // stream
        const int r = tid & 127;                 // row of the stream's tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + (uint32_t)(128 * st);
        const uint32_t tO0 = tmem + lanes + 256u;
        const float v_scale = p.v_scale;
        // sequences without a context: zeros for their nodes
        if (team == 0) {
            for (int s = cta; s < p.B; s += p.nctas) {
                const SeqInfo q = seq_info<TILES>(p, s, 0, false);
                if (q.L > 0 || q.n == 0) continue;
                const size_t e0 = (size_t)q.t0 * p.Hq * D, cnt = (size_t)q.n * p.Hq * D;
                const int es = p.out_f32 ? 4 : 2;
                uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + e0 * es);
                for (size_t i = tid; i < cnt * es / 16; i += 256) o[i] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        if (tid == 0) p.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
        int pc = 0, flat = misc[M_B0], joins = 0, stages = 0;
        bool ok = true;
        for (Walk<TILES> w(p, misc, team); ok && w.more(); w.next(p, team)) {
            const int seg = w.seg, buf = seg & 1, nc = w.chunks();
            const int r0 = team * TILES * kTile;
            const int rows = w.q.n * p.G - r0;   // rows of this team and those behind it
            const int copies = row_copies(rows);
            const bool idle = TILES == 2 && st == 1 && rows <= kTile;
            const int rt = (r & (kTile / copies - 1)) + (TILES == 2 ? st * kTile : 0);
            const bool warp_live = (rt & ~31) < rows;
            const bool in = rt < rows;
            const int node = in ? row_node(p, r0 + rt) : 0;
            const uint32_t* am = anc + (buf * kN + node) * 4;
            // the groups of 32 keys of a chunk that this warp's copy weighs
            const int gshare = 4 / copies, g_lo = (warp & 3) * copies / 4 * gshare, g_hi = g_lo + gshare;
            float m_ref = -INFINITY, l = 0.f;
            float sl2 = p.sl2;
            bool first = true;
            for (int c = TILES == 1 ? st : 0; c < nc && !idle; c += chunk_step(TILES)) {
                ok = wait_warp(bar(G::B_SFULL + st), (uint32_t)(pc & 1), misc);
                if (!ok) break;
                if (warp_live) {
                    umma::fence_after_sync();
                    if (FP8 && first)
                        sl2 = p.sl2 * reinterpret_cast<volatile float*>(gb + G::kQfacOff)[buf * TILES * kTile + (in ? rt : 0)];
                    const int np = w.chunk_pages(c);
                    const int p0 = (w.j + c * kPages) * kBlock;
                    const bool masked = np < kPages || w.drafted(c);
                    const int ng = (np + 1) / 2;         // groups of 32 keys
                    const int g_end = min(g_hi, ng);
                    // the keys of group g this row sees, as bits
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
                    // the largest scaled score of a group
                    auto group_max = [&](const uint32_t (&sr)[32], uint32_t vis) -> float {
                        float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        if (!masked && sl2 >= 0.f) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) a[k & 3] = fmaxf(a[k & 3], __uint_as_float(sr[k]));
                            return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * sl2;
                        }
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            a[k & 3] = fmaxf(a[k & 3], (vis >> k) & 1u ? __uint_as_float(sr[k]) * sl2 : -INFINITY);
                        return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
                    };
                    if (first) {
                        // the first chunk sets the reference maximum
                        float mx = -INFINITY;
                        for (int g = g_lo; g < g_end; ++g) {
                            uint32_t sr[32];
                            umma::tmem_ld32(tS + (uint32_t)(32 * g), sr);
                            umma::tmem_wait_ld();
                            mx = fmaxf(mx, group_max(sr, masked ? visible(g) : ~0u));
                        }
                        m_ref = mx;
                    }
                    float ls[4] = {0.f, 0.f, 0.f, 0.f};
                    // one group: its weights, in place of its scores
                    auto weigh = [&](const uint32_t (&sr)[32], int g) {
                        const uint32_t vis = masked ? visible(g) : ~0u;
                        const float gm = group_max(sr, vis);
                        // the reference moves only when it lags by more than 2^8; what
                        // was made with the old one is then scaled down in place
                        const bool move = in && gm > m_ref + kMaxLag;
                        if (__any_sync(kFull, move)) {
                            float alpha = 1.f;
                            if (move) {
                                alpha = ex2(m_ref - gm);     // 0 while nothing was seen
                                m_ref = gm;
                                l *= alpha;
#pragma unroll
                                for (int k = 0; k < 4; ++k) ls[k] *= alpha;
                            }
                            if (!first) {
#pragma unroll 1
                                for (int c0 = 0; c0 < D; c0 += 16) {
                                    uint32_t o[16];
                                    umma::tmem_ld16(tO0 + (uint32_t)(128 * st + c0), o);
                                    umma::tmem_wait_ld();
#pragma unroll
                                    for (int k = 0; k < 16; ++k)
                                        o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                                    umma::tmem_st16(tO0 + (uint32_t)(128 * st + c0), o);
                                }
                            }
#pragma unroll 1
                            for (int gg = g_lo; gg < g; ++gg) {
                                uint32_t h[16];
                                umma::tmem_ld16(tS + (uint32_t)(32 * gg), h);
                                umma::tmem_wait_ld();
                                if (FP8) {
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const __half2 x = *reinterpret_cast<const __half2*>(&h[e]);
                                        h[e] = pack_f16x2(__low2float(x) * alpha, __high2float(x) * alpha);
                                    }
                                } else {
                                    // the sum of the parts, scaled and split again
                                    uint32_t lw[16];
                                    umma::tmem_ld16(tS + (uint32_t)(32 * gg + 16), lw);
                                    umma::tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const float w0 = (bf16_lo(h[e]) + bf16_lo(lw[e])) * alpha;
                                        const float w1 = (bf16_hi(h[e]) + bf16_hi(lw[e])) * alpha;
                                        h[e] = pack_bf16x2(w0, w1);
                                        lw[e] = pack_bf16x2(w0 - bf16_lo(h[e]), w1 - bf16_hi(h[e]));
                                    }
                                    umma::tmem_st16(tS + (uint32_t)(32 * gg + 16), lw);
                                }
                                umma::tmem_st16(tS + (uint32_t)(32 * gg), h);
                            }
                        }
                        const float nm = (m_ref == -INFINITY ? 0.f : -m_ref) + (FP8 ? kBiasF16 : 0.f);
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float w0 = ex2(fmaf(__uint_as_float(sr[2 * e]), sl2, nm));
                            float w1 = ex2(fmaf(__uint_as_float(sr[2 * e + 1]), sl2, nm));
                            if (masked) {
                                w0 = (vis >> (2 * e)) & 1u ? w0 : 0.f;
                                w1 = (vis >> (2 * e + 1)) & 1u ? w1 : 0.f;
                            }
                            ls[e & 3] += w0 + w1;
                            if (FP8) {
                                hi[e] = pack_f16x2(w0, w1);
                            } else {
                                hi[e] = pack_bf16x2(w0, w1);
                                lo[e] = pack_bf16x2(w0 - bf16_lo(hi[e]), w1 - bf16_hi(hi[e]));
                            }
                        }
                        umma::tmem_st16(tS + (uint32_t)(32 * g), hi);
                        if (!FP8) umma::tmem_st16(tS + (uint32_t)(32 * g + 16), lo);
                    };
                    if (copies > 1) {
                        // the keys of the other copies weigh nothing here
                        uint32_t zero[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) zero[k] = 0u;
                        for (int g = 0; g < ng; ++g)
                            if (g < g_lo || g >= g_hi) {
                                umma::tmem_st16(tS + (uint32_t)(32 * g), zero);
                                if (!FP8) umma::tmem_st16(tS + (uint32_t)(32 * g + 16), zero);
                            }
                    }
                    // a group's scores are loaded while the one before is weighed
                    uint32_t next[32];
                    if (g_lo < g_end) umma::tmem_ld32(tS + (uint32_t)(32 * g_lo), next);
#pragma unroll 1
                    for (int g = g_lo; g < g_end; ++g) {
                        umma::tmem_wait_ld();
                        uint32_t sr[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) sr[k] = next[k];
                        if (g + 1 < g_end) umma::tmem_ld32(tS + (uint32_t)(32 * (g + 1)), next);
                        weigh(sr, g);
                    }
                    l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
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
            const bool whole = w.j == 0 && w.np == w.q.nb;
            // drafted V elements that were zeroed as infinities or NaN: added back for
            // the rows that see them
            auto add_back = [&](float* v, int cols, int c0, int of_node) {
                for (int k4 = 0; k4 < 4; ++k4) {
                    uint32_t b = 0u;
                    for (int q = 0; q < G::kPrepWarps; ++q) b |= badw[(buf * G::kPrepWarps + q) * 4 + k4];
                    for (b &= anc[(buf * kN + of_node) * 4 + k4]; b != 0u; b &= b - 1u) {
                        const int pos = w.q.base + 32 * k4 + __ffs(b) - 1;
                        const int blk = __ldg(p.bt + (size_t)w.s * p.max_blocks + pos / kBlock);
                        if (blk < 0 || blk >= p.num_blocks) continue;
                        const size_t at = (((size_t)blk * p.Hkv + w.h) * kBlock + pos % kBlock) * D + c0;
#pragma unroll
                        for (int k = 0; k < kStageCols; ++k) {
                            if (k >= cols) break;
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
            };
            bool back = false;                   // is there any such element?
            if (w.drafted(nc - 1))
                for (int q = 0; q < G::kPrepWarps * 4; ++q) back = back || badw[buf * G::kPrepWarps * 4 + q] != 0u;
            const size_t slot = (size_t)blockIdx.x * 2 + (w.j == 0 ? 1 : 0);
            // `cols` columns of one row, to the output or to the partials
            auto put = [&](float* v, auto cols, int c0, int row, float sum) {
                constexpr int N = decltype(cols)::value;
                const int nd = row_node(p, r0 + row);
                if (sum == 0.f) {
#pragma unroll
                    for (int k = 0; k < N; ++k) v[k] = 0.f;
                }
                if (back && !((padw[buf * 4 + (nd >> 5)] >> (nd & 31)) & 1u)) add_back(v, N, c0, nd);
                if (!whole) {
                    float* dst = p.part_o + (slot * (TILES * kTile) + row) * D + c0;
#pragma unroll
                    for (int k = 0; k < N; k += 2) *reinterpret_cast<float2*>(dst + k) = make_float2(v[k], v[k + 1]);
                    return;
                }
                const float inv = sum == 0.f ? 0.f : v_scale / sum;
                const size_t at = ((size_t)(w.q.t0 + nd) * p.Hq + (size_t)w.h * p.G + (r0 + row - nd * p.G)) * D + c0;
                if (p.out_f32) {
                    float* dst = static_cast<float*>(p.out) + at;
#pragma unroll
                    for (int k = 0; k < N; k += 2)
                        *reinterpret_cast<float2*>(dst + k) = make_float2(v[k] * inv, v[k + 1] * inv);
                } else {
                    uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
#pragma unroll
                    for (int k = 0; k < N; k += 2)
                        *reinterpret_cast<uint32_t*>(dst + k) = pack_bf16x2(v[k] * inv, v[k + 1] * inv);
                }
            };
            if (TILES == 1 || (copies > 1 && st == 0)) {
                // ---- join the partial results of a row: both streams' (TILES == 1),
                // all copies'
                float2* ml = reinterpret_cast<float2*>(gb + G::kMlOff);
                float* stage = reinterpret_cast<float*>(gb + G::kStageOff);
                ml[tid] = make_float2(m_ref, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(G::B_ML));
                ok = wait_warp(bar(G::B_ML), (uint32_t)(joins & 1), misc);
                if (!ok) break;
                ++joins;
                constexpr int streams = TILES == 1 ? 2 : 1;
                const int stride = kTile / copies;
                // largest maximum and joined sum of row `row`
                auto joined = [&](int row, float& M) -> float {
                    M = -INFINITY;
                    for (int i = 0; i < streams * copies; ++i)
                        M = fmaxf(M, ml[(i / copies) * kTile + (i % copies) * stride + row].x);
                    float sum = 0.f;
                    for (int i = 0; i < streams * copies; ++i) {
                        const float2 x = ml[(i / copies) * kTile + (i % copies) * stride + row];
                        sum += x.x == -INFINITY ? 0.f : x.y * ex2(x.x - M);
                    }
                    return sum;
                };
                float M;
                const float sum = joined(rt, M);
                const bool mine = nc > 1 || st == 0;     // did this stream have a chunk?
                const float a = m_ref == -INFINITY || !mine ? 0.f : ex2(m_ref - M);
                if (in && r == rt && st == 0 && !whole)
                    p.part_ml[slot * (TILES * kTile) + rt] = make_float2(M, sum);
                // kStageCols columns at a time through shared memory
                constexpr int T = G::kJoinWarps * 32;
                const int per = kStageCols * stride / T;         // columns of a thread: 2 .. 16
                const int row = tid * per / kStageCols, col = tid * per % kStageCols;
                float M2;
                const float sum2 = row < rows ? joined(row, M2) : 0.f;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += kStageCols) {
                    if (warp_live) {
                        uint32_t o[16];
                        umma::tmem_ld16(tO0 + (uint32_t)(128 * st + c0), o);
                        umma::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            stage[tid * kStageRow + k] = a == 0.f ? 0.f : __uint_as_float(o[k]) * a;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(G::B_STAGE));
                    ok = wait_warp(bar(G::B_STAGE), (uint32_t)(stages & 1), misc);
                    if (!ok) break;
                    ++stages;
                    if (row < rows) {
                        float v[kStageCols];
                        auto add = [&](auto cols) {
                            constexpr int N = decltype(cols)::value;
#pragma unroll
                            for (int k = 0; k < N; ++k) v[k] = 0.f;
                            for (int i = 0; i < streams * copies; ++i) {
                                const float* src = stage + ((i / copies) * kTile + (i % copies) * stride + row) * kStageRow + col;
#pragma unroll
                                for (int k = 0; k < N; ++k) v[k] += src[k];
                            }
                            put(v, cols, c0 + col, row, sum2);
                        };
                        if (per == 2) add(std::integral_constant<int, 2>());
                        else if (per == 4) add(std::integral_constant<int, 4>());
                        else add(std::integral_constant<int, 8>());
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(G::B_STAGE));
                    ok = wait_warp(bar(G::B_STAGE), (uint32_t)(stages & 1), misc);
                    if (!ok) break;
                    ++stages;
                }
                if (!ok) break;
            } else if (warp_live && !idle) {
                // ---- a row per thread, its whole result in one accumulator
                if (in && !whole) p.part_ml[slot * (TILES * kTile) + rt] = make_float2(m_ref, l);
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 16) {
                    uint32_t o[16];
                    umma::tmem_ld16(tO0 + (uint32_t)(128 * st + c0), o);
                    umma::tmem_wait_ld();
                    float v[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(o[k]);
                    if (in) put(v, std::integral_constant<int, 16>(), c0, rt, l);
                }
            }
            if (tid == 0 && w.j == 0 && !whole) {
                // the CTA with the first pages says where the partials are
                const int last = (int)(((long long)flat + w.q.nb - 1) / misc[M_Q]);
                p.meta[blockIdx.x] = make_int4(w.s, w.h, last - cta + 1, min(rows, TILES * kTile));
            }
            flat += w.np;
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(G::B_OFREE + buf));
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------- merge

// CTA (x, y): rows 8 y .. 8 y + 7 of the pair whose first partial CTA x of the
// split kernel wrote; one warp per row, the partials in CTA order.
constexpr int kMergeWarps = 8;

template <int D, int TILES>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_tree_merge_kernel(const TreeParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    const int4 meta = p.meta[blockIdx.x];
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
    const int parts = meta.z;
    if (parts <= 1 || row >= meta.w) return;
    constexpr int R = TILES * kTile, V = D / 32;
    // partial i of the pair: the first CTA's second slot, then the first slots
    auto slot = [&](int i) { return ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * R + row; };
    float M = -INFINITY;
    for (int i = lane; i < parts; i += 32) M = fmaxf(M, p.part_ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    float acc[V], l = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float2 ml = p.part_ml[slot(i)];
        const float* src = p.part_o + slot(i) * D + lane * V;
        float o[V];
        if constexpr (V == 4) {
            const float4 t = *reinterpret_cast<const float4*>(src);
            o[0] = t.x; o[1] = t.y; o[2] = t.z; o[3] = t.w;
        } else {
            const float2 t = *reinterpret_cast<const float2*>(src);
            o[0] = t.x; o[1] = t.y;
        }
        // a partial that saw nothing weighs nothing (its maximum is -inf)
        const float a = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
        l += ml.y * a;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += o[k] * a;
    }
    const float inv = l == 0.f ? 0.f : p.v_scale / l;
    const int team = blockIdx.x / p.nctas;
    const int r = team * R + row, node = row_node(p, r), g = r - node * p.G;
    int t0, n, bad;
    tree_span(p.starts, meta.x, p.total, p.max_nodes, t0, n, bad);
    const size_t at = ((size_t)(t0 + node) * p.Hq + (size_t)meta.y * p.G + g) * D + lane * V;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = l == 0.f ? 0.f : acc[k] * inv;
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

constexpr int kMinPages = 4;

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

// The tiles of a CTA, the teams and the workspace of a shape.
struct TreePlan {
    int tiles, teams, nctas;
    size_t part_o, part_ml, meta, total;
};

TreePlan tree_plan(int max_nodes, int G, int D)
{
    TreePlan t;
    const int rows = max_nodes * G;
    t.tiles = rows > kTile ? 2 : 1;
    t.teams = (rows + t.tiles * kTile - 1) / (t.tiles * kTile);
    t.nctas = num_sms_current() / t.teams;
    if (t.nctas < 1) t.nctas = 1;
    const size_t slots = (size_t)t.teams * t.nctas * 2 * t.tiles * kTile;
    t.part_o = 0;
    t.part_ml = up256(slots * D * sizeof(float));
    t.meta = t.part_ml + up256(slots * sizeof(float2));
    t.total = t.meta + up256((size_t)t.teams * t.nctas * sizeof(int4));
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

template <int D, bool FP8, int TILES>
int launch_tree(const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, cudaStream_t st)
{
    using G = Geo<D, FP8, TILES>;
    static bool ready[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return KV_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_tree_mu);
        if (!ready[dev]) {
            if (cudaFuncSetAttribute(paged_tree_kernel<D, FP8, TILES>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     G::kSmem) != cudaSuccess)
                return KV_ERR_CUDA;
            ready[dev] = true;
        }
    }
    const unsigned ctas = (unsigned)(p.teams * p.nctas);
    if (launch_pdl(paged_tree_kernel<D, FP8, TILES>, dim3(ctas), G::kThreads, G::kSmem, st, mk, mv,
                   p) != cudaSuccess)
        return KV_ERR_CUDA;
    const int rows = std::min(p.max_nodes * p.G, TILES * kTile);
    const dim3 grid(ctas, (unsigned)((rows + kMergeWarps - 1) / kMergeWarps));
    return launch_pdl(paged_tree_merge_kernel<D, TILES>, grid, kMergeWarps * 32, 0, st, p) ==
                   cudaSuccess
               ? KV_OK
               : KV_ERR_CUDA;
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
    if ((long long)num_seqs * max_blocks_per_seq * num_kv_heads >= INT_MAX ||
        (long long)num_blocks * num_kv_heads >= INT_MAX ||
        (long long)max_blocks_per_seq * kBlock >= INT_MAX)
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
    p.part_o = reinterpret_cast<float*>(ws + t.part_o);
    p.part_ml = reinterpret_cast<float2*>(ws + t.part_ml);
    p.meta = reinterpret_cast<int4*>(ws + t.meta);
    p.B = num_seqs;
    p.total = total_nodes;
    p.max_nodes = max_nodes;
    p.Hq = num_q_heads;
    p.Hkv = num_kv_heads;
    p.G = num_q_heads / num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.g_magic = p.G == 1 ? 0u : 0xffffffffu / (uint32_t)p.G + 1u;
    p.nctas = t.nctas;
    p.teams = t.teams;
    p.min_q = kMinPages;
    p.sl2 = scale * 1.4426950408889634f * (fp8 ? k_scale : 1.f);
    p.v_scale = fp8 ? v_scale : 1.f;
    p.out_f32 = out_dtype == KV_DTYPE_F32;
    p.test_stall = test_stall_cycles();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (head_dim == 128) {
        if (fp8)
            return t.tiles == 1 ? launch_tree<128, true, 1>(mk, mv, p, st)
                                : launch_tree<128, true, 2>(mk, mv, p, st);
        return t.tiles == 1 ? launch_tree<128, false, 1>(mk, mv, p, st)
                            : launch_tree<128, false, 2>(mk, mv, p, st);
    }
    if (fp8)
        return t.tiles == 1 ? launch_tree<64, true, 1>(mk, mv, p, st)
                            : launch_tree<64, true, 2>(mk, mv, p, st);
    return t.tiles == 1 ? launch_tree<64, false, 1>(mk, mv, p, st)
                        : launch_tree<64, false, 2>(mk, mv, p, st);
}
