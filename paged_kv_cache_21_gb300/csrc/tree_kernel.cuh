// What the kernels of paged_tree_attention share (paged_tree.cu, for trees of
// many query rows, and paged_tree_small.cu, for few): parameters, the cut of the
// work over CTAs, and the roles that bring queries, trees, keys and values into
// shared memory.
//
// A kernel's geometry G names its shared memory (offsets k..Off from a
// 1024-byte aligned base) and its barriers (B_..); both kernels consume K and V
// in chunks of up to 8 pages, chunk g of a CTA from slot g % slots of a ring of K
// and of one of V.  E4M3: the codes of K are multiplied as they are, with the
// query in three E5M2 parts; V is widened from a ring of codes to one of f16.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "paged_kv.h"
#include "tree_common.cuh"
#include "tree_launch.h"
#include "umma.cuh"

namespace pkv {

static __device__ DevErr g_tree_err;            // one per translation unit
static Launched g_launched;

namespace {

constexpr int kPages = 8;                       // pages of a chunk
constexpr int kKeys = kPages * kBlock;
constexpr int kN = KV_TREE_MAX_NODES;
constexpr int kRegion = kKeys * 128;            // one 128-byte column group of a chunk
constexpr long long kWaitLimit = 1LL << 31;     // ~1 s of SM clocks
constexpr float kMaxLag = 8.f;                  // the reference maximum may lag by 2^8
// f16 weights carry a factor of 2^7: at most 2^15 with the lag, and what f16
// rounds to zero is below 2^-31 of the largest weight
constexpr float kBiasF16 = 7.f;
// Up to this reference a weight's exponent is one fused operation, scale * score -
// reference.  The reference is a rounded product, so that the remainder for the very
// score it comes from, up to 2^-24 of it, is no more than 2^-3; above, where it would
// grow beyond what a weight can hold, products are rounded before.  (Always so: 16 nodes
// over E4M3 161 us for 149, 64 over bf16 329 for 320.)
constexpr float kFusedTo = 2097152.f;           // 2^21

// misc words: tensor-memory base; abort; the range: its first page's unit, pages, units
// per CTA, first sequence, KV head and page; chunks whose V is on its way (bf16)
enum Misc { M_TMEM = 0, M_ABORT, M_B0, M_CNT, M_Q, M_S0, M_H0, M_J0, M_VISSUED };

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
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

// Wait until the V of chunk g is on its way into its slot.  The warp that fixes V
// rows, which does not follow every chunk of the ring, does this before it waits for
// the chunk's barrier: the slot's previous phase is then known to be over, and the
// phase's parity to be that of chunk g.
__device__ __forceinline__ bool wait_issued(int g, volatile int* misc)
{
    if (misc[M_VISSUED] > g) return true;
    const long long t0 = clock64();
    while (misc[M_VISSUED] <= g) {
        if (misc[M_ABORT]) return false;
        if (clock64() - t0 > kWaitLimit) {
            misc[M_ABORT] = 1;
            raise_flag(&g_tree_err, KV_DEVERR_PIPELINE_TIMEOUT, blockIdx.x);
            return false;
        }
    }
    return true;
}

// wait_bar for a whole warp.
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

// One sequence as a team of CTAs sees it.
struct SeqInfo {
    int t0, n, L, base, nb;     // nb: pages, 0 when the team has no rows here
};

// `first_row`: the team's first row of a KV head's n * G rows.
__device__ __forceinline__ SeqInfo seq_info(const TreeParams& p, int s, int first_row, bool flag)
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
    const int rows = q.n * p.G;
    q.L = L;
    q.base = L > q.n ? L - q.n : 0;
    q.nb = rows > first_row && rows > p.rows_above && rows <= p.rows_to ? (L + kBlock - 1) / kBlock : 0;
    return q;
}

// Does a node that is not padding see any position?  `am`: the nodes it sees, as bits.
// (A row that does, and whose weights sum to nothing, had scores of -inf alone: its
// softmax is NaN.)
template <int WORDS>
__device__ __forceinline__ bool sees_any(const SeqInfo& q, const uint32_t* am)
{
    bool any = q.base > 0;
    for (int k = 0; k < WORDS; ++k) {
        const int lim = q.L - 32 * k;            // (nodes there is no room for are not cached)
        if (lim > 0) any = any || (lim < 32 ? am[k] & ((1u << lim) - 1u) : am[k]) != 0u;
    }
    return any;
}

// Node (within the sequence) of row r of a KV head's rows.
__device__ __forceinline__ int row_node(const TreeParams& p, int r)
{
    return p.g_magic ? (int)__umulhi((uint32_t)r, p.g_magic) : r;
}

// One ring that the MMAs read: chunk g's slot, its barriers and their parity.  The
// barriers that say a chunk's slot may be refilled may be more than the slots.
template <int SLOTS, int FULL, int FREE, int FREES = SLOTS>
struct Ring {
    static constexpr int kSlots = SLOTS;
    static_assert(FREES >= SLOTS, "a slot's release is seen before the barrier's next phase");
    static __device__ __forceinline__ int slot(int g) { return (int)((uint32_t)g % SLOTS); }
    static __device__ __forceinline__ uint32_t parity(int g) { return (uint32_t)g / SLOTS & 1u; }
    static __device__ __forceinline__ int full(int g) { return FULL + slot(g); }
    static __device__ __forceinline__ int free(int g) { return FREE + (int)((uint32_t)g % FREES); }
    static __device__ __forceinline__ uint32_t free_parity(int g) { return (uint32_t)g / FREES & 1u; }
};

// The segments of a CTA's range: the pages [j, j + np) of one (sequence, KV
// head) each.  Every role walks the same list.
struct Walk {
    int s, h, j, rem, seg, np;
    SeqInfo q;
    __device__ __forceinline__ Walk(const TreeParams& p, const volatile int* misc, int first_row)
    {
        s = misc[M_S0];
        h = misc[M_H0];
        j = misc[M_J0];
        rem = misc[M_CNT];
        seg = 0;
        np = 0;
        if (rem > 0) {
            q = seq_info(p, s, first_row, false);
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
    // the chunks before the first that is not whole or reaches them
    __device__ __forceinline__ int plain_chunks() const
    {
        return max(0, min(np, q.base / kBlock - j) / kPages);
    }
    __device__ __forceinline__ bool whole() const { return j == 0 && np == q.nb; }
    __device__ __forceinline__ void next(const TreeParams& p, int first_row)
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
                q = seq_info(p, s, first_row, false);
            } while (q.nb == 0);
        }
        np = min(q.nb, rem);
    }
};

// This CTA's range of its team's list of pages, by sequence and KV head: equal
// shares of at least p.min_q units, where a page is a unit and each (sequence, KV
// head) costs kExtraPages more before its first page (its queries, tree and results), so
// that CTAs with many short sequences get fewer pages.  One warp.
__device__ __forceinline__ void cut_work(const TreeParams& p, volatile int* misc, int first_row, int cta,
                                         bool flag, int lane)
{
    long long total = 0;
    for (int b = 0; b < p.B; b += 32) {
        int nb = 0;
        if (b + lane < p.B) nb = seq_info(p, b + lane, first_row, flag).nb;
        total += warp_sum_ll(nb > 0 ? nb + kExtraPages : 0);
    }
    total *= p.Hkv;
    long long q = (total + p.nctas - 1) / p.nctas;
    if (q < p.min_q) q = p.min_q;
    // the first page at or behind unit x: its sequence, head and index, its unit, and
    // how many pages are before it
    struct At {
        int s, h, j;
        long long unit, pages;
    };
    const long long lo = min((long long)cta * q, total), hi = min(lo + q, total);
    At at[2] = {{0, 0, 0, 0, 0}, {0, 0, 0, 0, 0}};
    bool found[2] = {false, false};
    long long units = 0, pages = 0;              // up to the 32 sequences at hand
    for (int b = 0; b < p.B && !(found[0] && found[1]); b += 32) {
        int nb = 0;
        if (b + lane < p.B) nb = seq_info(p, b + lane, first_row, false).nb;
        const long long u = nb > 0 ? (long long)(nb + kExtraPages) * p.Hkv : 0, n = (long long)nb * p.Hkv;
        long long iu = u, in = n;
        for (int o = 1; o < 32; o <<= 1) {
            const long long tu = __shfl_up_sync(kFull, iu, o), tn = __shfl_up_sync(kFull, in, o);
            if (lane >= o) {
                iu += tu;
                in += tn;
            }
        }
        iu += units;
        in += pages;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const long long x = e == 0 ? lo : hi;
            const unsigned m = __ballot_sync(kFull, iu > x);
            if (found[e] || !m) continue;
            found[e] = true;
            const int src = __ffs(m) - 1;
            const int nbs = __shfl_sync(kFull, nb, src), v = nbs + kExtraPages;
            const long long before = __shfl_sync(kFull, iu - u, src);
            const int off = (int)(x - before), h = off / v, j = max(0, off - h * v - kExtraPages);
            at[e] = {b + src, h, j, before + (long long)h * v + kExtraPages + j,
                     __shfl_sync(kFull, in - n, src) + (long long)h * nbs + j};
        }
        units = __shfl_sync(kFull, iu, 31);
        pages = __shfl_sync(kFull, in, 31);
    }
    if (!found[1]) at[1].pages = pages;          // (hi is the end of the list)
    if (lane == 0) {
        misc[M_B0] = (int)at[0].unit;
        misc[M_CNT] = found[0] ? (int)(at[1].pages - at[0].pages) : 0;
        misc[M_Q] = (int)q;
        misc[M_S0] = at[0].s;
        misc[M_H0] = at[0].h;
        misc[M_J0] = at[0].j;
    }
}

// Byte offset of 16-byte chunk c of row r in a [128 rows x 128 B] region
// (128-byte swizzle).
__device__ __forceinline__ uint32_t region_off(int r, int c)
{
    return (uint32_t)(r * 128) + (uint32_t)(((c ^ (r & 7)) & 7) * 16);
}

// Four E4M3 codes as four f16: exact.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t x, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
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

// Role of a warp: K (WHICH 0), V (1) or both (2) of every chunk by TMA.  A warp
// issues one copy in ~80 clocks (measured: 26 bytes a clock in 2 KB boxes, twice
// that from two warps), less than an SM's share of HBM at its usual clock, so
// where K and V come fast each has a warp of its own.
template <class G, int WHICH>
__device__ __forceinline__ void copy_role(const TreeParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                          uint32_t sb, volatile int* misc, int first_row, int lane)
{
    constexpr bool FP8 = G::kFp8;
    constexpr int kPage = FP8 ? G::kPageBytes : kBlock * 128;    // bytes of a box
    auto bar = [&](int i) -> uint32_t { return sb + (uint32_t)(G::kBarOff + 8 * i); };
    const uint64_t pol = l2_evict_first_policy();
    const int box = FP8 ? 0 : lane % G::kBoxes, page = FP8 ? lane : lane / G::kBoxes;
    int gk = 0, gv = 0;                          // chunks issued
    // this lane's page of a chunk, its KV head; the pages to copy
    struct Pages {
        int z, n;
        bool mine;
    };
    auto issue = [&](auto ring, int off, int slot_bytes, const CUtensorMap& tm, int& g, const Pages& c) -> bool {
        using R = decltype(ring);
        if (g >= R::kSlots && !wait_warp(bar(R::free(g - R::kSlots)), R::free_parity(g - R::kSlots), misc))
            return false;
        const uint32_t fb = bar(R::full(g));
        if (lane == 0) {
            if (c.n > 0) mbar_arrive_expect_tx(fb, (uint32_t)(c.n * G::kPageBytes));
            else mbar_arrive(fb);
        }
        __syncwarp();
        if (c.mine) {
            const uint32_t dst = sb + (uint32_t)(off + R::slot(g) * slot_bytes + box * kRegion + page * kPage);
            if (p.teams == 1)                    // read once: first out of L2
                tma_load_3d_hint(dst, &tm, box * 64, 0, c.z, fb, pol);
            else
                tma_load_3d(dst, &tm, box * 64, 0, c.z, fb);
        }
        ++g;
        return true;
    };
    auto issue_k = [&](const Pages& c) {
        return issue(typename G::KRing(), G::kKOff, G::kLoadBytes, tm_k, gk, c);
    };
    auto issue_v = [&](const Pages& c) {
        if (!issue(typename G::VLoad(), G::kVLoadOff, G::kLoadBytes, tm_v, gv, c)) return false;
        if (!FP8 && lane == 0) misc[M_VISSUED] = gv;
        return true;
    };
    bool ok = true, held = false;                // (a warp for both: V comes a chunk after K)
    Pages before = {0, 0, false};
    for (Walk w(p, misc, first_row); ok && w.more(); w.next(p, first_row)) {
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
            const int my = __shfl_sync(kFull, ids, (c & 3) * kPages + page % kPages);
            const bool in = page < w.chunk_pages(c);
            Pages now;
            now.mine = in && my >= 0 && my < p.num_blocks;
            now.z = my * p.Hkv + w.h;
            if (WHICH != 1 && in && !now.mine && box == 0) raise_flag(&g_tree_err, KV_DEVERR_BLOCK_OUT_OF_RANGE, my);
            now.n = __popc(__ballot_sync(kFull, now.mine && box == 0));
            if (WHICH != 1) ok = issue_k(now);
            if (ok && WHICH == 1) ok = issue_v(now);
            if (ok && WHICH == 2 && held) ok = issue_v(before);
            before = now;
            held = true;
        }
    }
    if (ok && WHICH == 2 && held) issue_v(before);
    // every issued copy lands before the CTA can end
    if (lane == 0) {
        for (int i = gk > G::KRing::kSlots ? gk - G::KRing::kSlots : 0; i < gk; ++i)
            mbar_wait_bounded(bar(G::KRing::full(i)), G::KRing::parity(i), kWaitLimit);
        for (int i = gv > G::VLoad::kSlots ? gv - G::VLoad::kSlots : 0; i < gv; ++i)
            mbar_wait_bounded(bar(G::VLoad::full(i)), G::VLoad::parity(i), kWaitLimit);
    }
    __syncwarp();
}

// The nodes each node of the segment's tree sees, as bits, by doubling along the
// parents; and which nodes are padding.  One warp.
template <class G>
__device__ __forceinline__ void tree_masks(const TreeParams& p, const Walk& w, uint8_t* gb, int lane)
{
    constexpr int W = G::kWords;             // words of bits: a tree here has at most 32 W nodes
    const int buf = w.seg & 1, n = w.q.n;
    uint32_t* anc = reinterpret_cast<uint32_t*>(gb + G::kAncOff);
    volatile uint32_t* padw = reinterpret_cast<volatile uint32_t*>(gb + G::kPadOff);
    volatile int* ptr = reinterpret_cast<volatile int*>(gb + G::kPtrOff);
    volatile uint32_t* am = anc + buf * 32 * W * W;
    int up[W];
    uint32_t m[W][W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
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
        for (int v = 0; v < W; ++v)
            m[k][v] = v == k && i < n && !pad ? 1u << lane : 0u;
    }
    for (int reach = 1; reach < n; reach *= 2) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const int i = 32 * k + lane;
            ptr[i] = up[k];
#pragma unroll
            for (int v = 0; v < W; ++v) am[W * i + v] = m[k][v];
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < W; ++k) {
            if (up[k] >= 0) {
                const int a = up[k];
#pragma unroll
                for (int v = 0; v < W; ++v) m[k][v] |= am[W * a + v];
                up[k] = ptr[a];
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int v = 0; v < W; ++v) am[W * (32 * k + lane) + v] = m[k][v];
}

// Zero the V rows behind the context, and the infinities and NaN of the drafted
// rows, of the segment's chunks that reach the drafted positions (bf16).  One
// warp.  False: given up.
template <class G>
__device__ __forceinline__ bool fix_values(const TreeParams& p, const Walk& w, uint32_t sb, uint8_t* gb,
                                           volatile int* misc, int g0, int lane)
{
    auto bar = [&](int i) -> uint32_t { return sb + (uint32_t)(G::kBarOff + 8 * i); };
    volatile uint32_t* badw = reinterpret_cast<volatile uint32_t*>(gb + G::kBadOff);
    constexpr int D = G::kD, C = D / 8, RI = 32 / C, pw = 0;
    const int buf = w.seg & 1, nc = w.chunks(), c = lane % C;
    bool ok = true;
    // ---- V rows of the chunks that reach the drafted positions
    for (int ch = 0; ok && ch < nc; ++ch) {
        if (!w.drafted(ch)) continue;
        const int gv = g0 + ch;
        ok = __all_sync(kFull, wait_issued(gv, misc)) &&
             wait_warp(bar(G::VRing::full(gv)), G::VRing::parity(gv), misc);
        if (!ok) break;
        const uint32_t vb = sb + (uint32_t)(G::kVOff + G::VRing::slot(gv) * G::kSlot);
        const int p0 = (w.j + ch * kPages) * kBlock;
        const int lo = max(0, w.q.base - p0), hi = w.chunk_pages(ch) * kBlock;
        for (int rb = lo; rb < hi; rb += RI) {
            const int r = rb + lane / C;
            const uint32_t at = vb + (uint32_t)((c >> 3) * kRegion) + region_off(r & 127, c & 7);
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
        if (lane == 0) mbar_arrive(bar(G::B_FIX + G::VRing::slot(gv)));
    }
    return ok;
}

// Widen the E4M3 codes of the segment's V to f16, with what fix_values does on the
// way.  One of the prep warps (pw).  False: given up.
template <class G>
__device__ __forceinline__ bool widen(const TreeParams& p, const Walk& w, uint32_t sb, uint8_t* gb,
                                      volatile int* misc, int g0, int pw, int lane)
{
    using L = typename G::VLoad;
    using R = typename G::VRing;
    auto bar = [&](int i) -> uint32_t { return sb + (uint32_t)(G::kBarOff + 8 * i); };
    volatile uint32_t* badw = reinterpret_cast<volatile uint32_t*>(gb + G::kBadOff);
    constexpr int D = G::kD;
    const int buf = w.seg & 1, nc = w.chunks();
    // 16 codes a thread and step: piece cc of row r.  Eight lanes that go to
    // shared memory together have eight rows, so their pieces lie, swizzled, in
    // different banks on both sides; a step is RS rows, a multiple of the swizzle's
    // period, so that offsets between steps are constants.
    constexpr int CR = D / 16;               // 16-code pieces of a row
    constexpr int RS = G::kPrepWarps * 32 / CR;      // rows of the warps' step
    constexpr int kSteps = kKeys / RS;
    const int t = pw * 32 + lane;
    const int r0 = t % RS, cc = t / RS;
    // the copy's swizzle: 16-byte pieces XOR bits 7 and up of the address
    const uint32_t flat = (uint32_t)(r0 * D + cc * 16);
    const uint32_t src0 = flat ^ (((flat >> 7) & (D == 128 ? 7u : 3u)) << 4);
    const uint32_t dst0 = (uint32_t)((cc >> 2) * kRegion) + region_off(r0, (2 * cc) & 7);
    const uint32_t dst1 = (uint32_t)((cc >> 2) * kRegion) + region_off(r0, (2 * cc + 1) & 7);
    for (int ch = 0; ch < nc; ++ch) {
        const int g = g0 + ch;
        if (!wait_warp(bar(L::full(g)), L::parity(g), misc)) return false;
        if (g >= R::kSlots && !wait_warp(bar(R::free(g - R::kSlots)), R::free_parity(g - R::kSlots), misc))
            return false;
        const uint32_t raw = sb + (uint32_t)(G::kVLoadOff + L::slot(g) * G::kLoadBytes) + src0;
        const uint32_t dst = sb + (uint32_t)(G::kVOff + R::slot(g) * G::kSlot);
        auto store = [&](int step, const uint32_t (&v)[4]) {
            uint4 a, b;
            e4m3x4_to_f16x4(v[0], a.x, a.y);
            e4m3x4_to_f16x4(v[1], a.z, a.w);
            e4m3x4_to_f16x4(v[2], b.x, b.y);
            e4m3x4_to_f16x4(v[3], b.z, b.w);
            sts128(dst + dst0 + (uint32_t)(step * RS * 128), a);
            sts128(dst + dst1 + (uint32_t)(step * RS * 128), b);
        };
        const int keys = w.chunk_pages(ch) * kBlock;
        if (keys == kKeys && !w.drafted(ch)) {
#pragma unroll
            for (int s0 = 0; s0 < kSteps; s0 += 4) {     // four loads in flight
                uint32_t v[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) lds128(v[k], raw + (uint32_t)((s0 + k) * RS * D));
#pragma unroll
                for (int k = 0; k < 4; ++k) store(s0 + k, v[k]);
            }
        } else {
            for (int step = 0; step * RS + r0 < keys; ++step) {
                const int pos = (w.j + ch * kPages) * kBlock + step * RS + r0;
                uint32_t v[4];
                lds128(v, raw + (uint32_t)(step * RS * D));
                if (pos >= w.q.L) {
                    v[0] = v[1] = v[2] = v[3] = 0u;
                } else if (pos >= w.q.base && drop_non_finite<true>(v)) {
                    const int an = pos - w.q.base;
                    atomicOr(const_cast<uint32_t*>(&badw[(buf * G::kPrepWarps + pw) * 4 + (an >> 5)]),
                             1u << (an & 31));
                }
                store(step, v);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bar(L::free(g)));
            mbar_arrive(bar(R::full(g)));
        }
    }
    return true;
}

// A query row's 8 elements (16 bytes of bf16) as three E5M2 parts, for E4M3 keys:
// the row is scaled by a power of two that brings its largest |element| into
// [2^14, 2^15).  As f16 an element is then exact down to 2^-17; E5M2 is an f16's upper
// byte, so that a part is what the ones before leave with its lower byte cleared, three
// bits.  Three parts hold bf16's eight bits exactly, down to 2^-24 of the row's
// largest element (2^-9 here); below, where parts fall between E5M2's steps of
// 2^-16, an element loses at most 2^-16, 2^-30 of the largest.  (Two parts of
// E4M3, four bits each but steps of 2^-9, were exact down to 2^-10 of the largest
// only: an outlier cost the other elements theirs.  32 x 8192 tokens, 4 heads: 8 nodes 117
// us then, 121 now; 16 nodes 153, 156; 64 nodes 388, 434.)  The scores are
// multiplied by `up` again.  A row with infinities or NaN has up = NaN.  The row's
// D / 8 lanes call together.
constexpr int kQueryParts = 3;

template <int D>
__device__ __forceinline__ void query_e5m2(uint4 v, uint2 (&parts)[kQueryParts], float& up)
{
    const uint32_t q4[4] = {v.x, v.y, v.z, v.w};
    uint32_t big = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) big = max(big, max(q4[k] & 0x7fffu, (q4[k] >> 16) & 0x7fffu));
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(kFull, big, o));
    // (both powers are normal floats; the smallest bf16 is 2^-7 at 2^126 times its value)
    const int e = big == 0 ? 0 : max((int)(big >> 7) - (127 + 14), -126);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    up = big >= 0x7f80u ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)(127 + e) << 23);
    uint32_t p[kQueryParts][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t x = pack_f16x2(bf16_lo(q4[k]) * down, bf16_hi(q4[k]) * down);
#pragma unroll
        for (int part = 0; part < kQueryParts; ++part) {
            p[part][k] = x & 0xff00ff00u;
            const __half2 left = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&p[part][k]));
            x = *reinterpret_cast<const uint32_t*>(&left);
        }
    }
#pragma unroll
    for (int part = 0; part < kQueryParts; ++part)
        parts[part] = make_uint2(__byte_perm(p[part][0], p[part][1], 0x7531), __byte_perm(p[part][2], p[part][3], 0x7531));
}

// Byte offset of byte 8 c of row r of a tile of D-byte rows, with the swizzle that
// the copies give the codes (128 bytes at D = 128, 64 at 64).
template <int D>
__device__ __forceinline__ uint32_t code_off(int r, int c)
{
    const uint32_t a = (uint32_t)(r * D + 8 * c);
    return a ^ (((a >> 7) & (D == 128 ? 7u : 3u)) << 4);
}

// Descriptor of a K-major tile of E4M3 rows as the copies leave it.
template <int D>
__device__ __forceinline__ uint64_t code_desc(uint32_t saddr)
{
    return D == 128 ? umma::smem_desc_sw128(saddr, 16, 1024) : umma::smem_desc_sw64(saddr, 16, 512);
}

// Sequences without a context get zeros for their nodes (threads 0 .. nthreads - 1
// of the CTAs of the kernel that does it).
__device__ __forceinline__ void zero_empty(const TreeParams& p, int D, int cta, int ctas, int tid, int nthreads)
{
    for (int s = cta; s < p.B; s += ctas) {
        const SeqInfo q = seq_info(p, s, 0, false);
        if (q.L > 0 || q.n == 0) continue;
        const size_t e0 = (size_t)q.t0 * p.Hq * D, cnt = (size_t)q.n * p.Hq * D;
        const int es = p.out_f32 ? 4 : 2;
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + e0 * es);
        for (size_t i = tid; i < cnt * es / 16; i += nthreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace
}  // namespace pkv
