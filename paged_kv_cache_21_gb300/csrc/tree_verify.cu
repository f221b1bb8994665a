// kv_tree_verify: which nodes of each sequence's draft tree the target accepts,
// from given uniform numbers, and the token after the last of them.
//
// The walk itself is a few dozen comparisons; what costs is the rows of vocab
// probabilities.  At the node where the walk stops, the remaining distribution
//     R_j = max(p_j - a q_j, 0)
// has to be summed and then cut at u * sum R, and before that once for every
// refused child but the last.  (R of the j-th refusal in closed form: with
// Z = sum R, the next residual max(R / Z - q, 0) is proportional to
// max(p - (a + Z) q, 0), so one number `a` carries all refusals of a node.)
//
// What decides the result is a comparison with a cumulative sum over up to
// hundreds of thousands of entries, so the sums must be far finer than the
// entries' spacing in them: float32 would move one sampled token in a few dozen.
// Each thread sums in pairs of floats (a sum and its rounding error: 2^-46), and
// so do the joins over threads and CTAs: this GPU's double precision units would
// take ten times as long.  Two entries go through one packed instruction.
//
// One cluster of CTAs serves a sequence: each CTA takes a contiguous slice of
// the row, its warps contiguous sub-slices, and the CTAs exchange their sums
// through distributed shared memory.  All CTAs walk the tree in step, from
// copies of the tree and of the single probabilities at the drafted tokens
// (gathered at once, for all nodes) in shared memory.  The CTA, warp and lane
// that hold the cut then find the token; the row comes from L2 by then.  The
// cluster is as large as lets all sequences run at once, two CTAs an SM.
//
// Measured: 64 trees of 26 nodes, 128000 float32 entries: 54 us, where the rows of
// the last nodes take 9.6 at HBM's rate.  The sequence with the most refusals sums
// five times in turn, ~9.5K clocks each: 256 KB a CTA and pass through its SM's
// share of L2 bandwidth (two CTAs, 53 of ~64 bytes a clock), ~17 packed operations
// for two entries beside it.  Clusters of 8 do not run all at once (61 us), more
// but smaller CTAs are slower too (63); one chain of 5, 32000 entries: 8.2 us, of
// launch, tree and one pass.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <utility>

#include "device_common.cuh"
#include "internal.h"
#include "paged_kv.h"
#include "tree_common.cuh"

namespace cg = cooperative_groups;

namespace pkv {

__device__ DevErr g_verify_err;
static Launched g_launched;

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr int kMaxCluster = 8;           // the portable cluster size
constexpr int kN = KV_TREE_MAX_NODES;

struct VerifyParams {
    int32_t* lens;
    int32_t* nodes;
    int32_t* out;
    const void* target;
    const void* draft;                   // null: drafted tokens are certain
    long long target_stride, draft_stride;
    const int32_t* tokens;
    const int32_t* parents;
    const int32_t* starts;
    const float* accept_u;
    const float* sample_u;
    int total, max_nodes, vocab, greedy;
};

// ------------------------------------------------------------- pairs of floats

// A sum and its rounding error.
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair add(Pair a, Pair b)
{
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
    const float h = s + e;
    return {h, e - (h - s)};
}

__device__ __forceinline__ bool above(Pair a, Pair b) { return (a.hi - b.hi) + (a.lo - b.lo) > 0.f; }

__device__ __forceinline__ Pair mul(Pair a, float b)
{
    const float h = __fmul_rn(a.hi, b), e = fmaf(a.hi, b, -h) + a.lo * b, r = h + e;
    return {r, e - (r - h)};
}

__device__ __forceinline__ Pair mul(Pair a, Pair b)
{
    const float h = __fmul_rn(a.hi, b.hi), e = fmaf(a.hi, b.hi, -h) + (a.hi * b.lo + a.lo * b.hi), r = h + e;
    return {r, e - (r - h)};
}

__device__ __forceinline__ Pair shfl(Pair v, int src)
{
    return {__shfl_sync(kFull, v.hi, src), __shfl_sync(kFull, v.lo, src)};
}

__device__ __forceinline__ Pair warp_sum(Pair v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = add(v, Pair{__shfl_xor_sync(kFull, v.hi, o), __shfl_xor_sync(kFull, v.lo, o)});
    return v;
}

// Sums up to and with each lane.
__device__ __forceinline__ Pair warp_scan(Pair v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair up = {__shfl_up_sync(kFull, v.hi, o), __shfl_up_sync(kFull, v.lo, o)};
        if (lane >= o) v = add(up, v);
    }
    return v;
}

// Two running sums side by side: x plus its error xe, for two entries.
struct Sum2 {
    u64 hi = 0ull, lo = 0ull;
    __device__ __forceinline__ void add(u64 x, u64 xe)
    {
        const u64 s = add2(hi, x), b = sub2(s, hi);
        lo = add2(lo, add2(add2(sub2(hi, sub2(s, b)), sub2(x, b)), xe));
        hi = s;
    }
    __device__ __forceinline__ void add(u64 x)
    {
        const u64 s = add2(hi, x), b = sub2(s, hi);
        lo = add2(lo, add2(sub2(hi, sub2(s, b)), sub2(x, b)));
        hi = s;
    }
    __device__ __forceinline__ Pair value() const
    {
        float h0, h1, l0, l1;
        unpack2(hi, h0, h1);
        unpack2(lo, l0, l1);
        return pkv::add(Pair{h0, l0}, Pair{h1, l1});
    }
};

// ------------------------------------------------------------------- weights

// What counts as zero: negative, infinite and NaN entries.
__device__ __forceinline__ float clean(float x) { return x > 0.f && x < INFINITY ? x : 0.f; }

template <bool BF16>
__device__ __forceinline__ float load1(const void* row, long long i)
{
    if (BF16) return __uint_as_float((uint32_t)__ldg((const uint16_t*)row + i) << 16);
    return __ldg((const float*)row + i);
}

// VEC consecutive entries: one 16-byte load, or one entry.
template <bool BF16, int VEC>
__device__ __forceinline__ void loadv(const void* row, long long i, float (&x)[VEC])
{
    if constexpr (VEC == 1) {
        x[0] = load1<BF16>(row, i);
    } else if constexpr (BF16) {
        const uint4 w = __ldg((const uint4*)((const uint16_t*)row + i));
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = bf16_lo(v[k]);
            x[2 * k + 1] = bf16_hi(v[k]);
        }
    } else {
        const float4 w = __ldg((const float4*)((const float*)row + i));
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    }
}

// The remaining weights of a node: R_j = max(p_j - a q_j, 0) with a = ah + al, the
// product and the difference exact but for 2^-46; or p_j without the refused tokens.
struct Weights {
    const void* p;
    const void* q;                       // null: no refusal with a draft
    float ah, al;
    const int* gone;                     // refused tokens (no draft)
    int ngone;

    // one entry, by scalars
    __device__ __forceinline__ Pair one(int i, float x, float y) const
    {
        x = clean(x);
        for (int g = 0; g < ngone; ++g)
            if (gone[g] == i) x = 0.f;
        if (!q) return {x, 0.f};
        y = clean(y);
        const float ph = __fmul_rn(ah, y);       // not to be contracted into the difference
        const float pe = fmaf(ah, y, -ph) + al * y;
        const float s = x - ph, b = s - x;
        const float e = ((x - (s - b)) + (-ph - b)) - pe;
        return s + e > 0.f ? Pair{s, e} : Pair{0.f, 0.f};
    }
    // two entries into a sum, for entries of q that are finite and not negative (a
    // negative or NaN entry of p adds nothing; an infinite one makes the sum so)
    __device__ __forceinline__ void two(u64 x, u64 y, Sum2& sum) const
    {
        const u64 nph = mul2(pack2(-ah, -ah), y);
        const u64 pe = fma2(pack2(al, al), y, fma2(pack2(ah, ah), y, nph));
        // (the sum's rounding error this way needs x >= a y: so it is where s > 0)
        const u64 s = add2(x, nph), e = sub2(sub2(nph, sub2(s, x)), pe);
        float s0, s1, e0, e1;
        unpack2(s, s0, s1);
        unpack2(e, e0, e1);
        sum.add(pack2(fmaxf(s0, 0.f), fmaxf(s1, 0.f)), pack2(s0 > 0.f ? e0 : 0.f, s1 > 0.f ? e1 : 0.f));
    }
};

// Shared state of a CTA.  Every CTA of a cluster holds the same tree and walk.
struct Shared {
    int par[kN], tok[kN], child[kN], sibling[kN];    // first child and next sibling, -1: none
    float pv[kN], qv[kN], u[kN];         // p and q of the node's token at its parent
    bool takes[kN];                      // accepted as its parent's first child
    int gone[kN];                        // refused tokens of the node (no draft)
    int path[kN];
    Pair sums[2][kMaxCluster * kWarps];  // of every warp of the cluster
    float best[2][kMaxCluster];          // greedy: largest entry and where it is
    int best_at[2][kMaxCluster];
    float wbest[kWarps];
    int wbest_at[kWarps];
    Pair a, Z;
    int v, next_child, ngone, depth, state, n, t0, token;
};

enum State { kWalk, kNeedSum, kDone };

// The slice [lo, hi) of warp w of nw: `lead` entries before the first whole vector
// (the first warp's), then steps of 32 vectors, spread evenly.
__device__ __forceinline__ void warp_slice(int vocab, int lead, int vec, int w, int nw, int& lo,
                                           int& hi)
{
    const int step = 32 * vec;
    const int body = vocab > lead ? vocab - lead : 0;
    const int units = (body + step - 1) / step;
    const int u0 = (int)((long long)units * w / nw), u1 = (int)((long long)units * (w + 1) / nw);
    lo = w == 0 ? 0 : lead + u0 * step;
    hi = min(vocab, lead + u1 * step);
    if (lo > hi) lo = hi;
}

// Every entry of [lo, hi), lanes side by side: whole vectors to `vec(i, x, y)`, the
// entries before and after them to `one(i, x, y)`.
template <bool BF16, int VEC, typename FV, typename F1>
__device__ __forceinline__ void for_slice(const void* p, const void* q, int lead, int lo, int hi,
                                          int lane, FV&& vec, F1&& one)
{
    int i = lo;
    if (VEC > 1 && lo == 0 && lead > 0) {
        if (lane < lead && lane < hi) one(lane, load1<BF16>(p, lane), q ? load1<BF16>(q, lane) : 0.f);
        i = lead;
    }
    if (q) {
#pragma unroll 4
        for (int at = i + lane * VEC; at + VEC <= hi; at += 32 * VEC) {
            float x[VEC], y[VEC];
            loadv<BF16, VEC>(p, at, x);
            loadv<BF16, VEC>(q, at, y);
            vec(at, x, y);
        }
    } else {
#pragma unroll 4
        for (int at = i + lane * VEC; at + VEC <= hi; at += 32 * VEC) {
            float x[VEC];
            loadv<BF16, VEC>(p, at, x);
            vec(at, x, x);
        }
    }
    if (VEC > 1 && hi > i) {
        const int tail = (hi - i) % VEC, at = hi - tail + lane;
        if (lane < tail) one(at, load1<BF16>(p, at), q ? load1<BF16>(q, at) : 0.f);
    }
}

// Sum of the weights of this thread's entries of [lo, hi).
template <bool BF16, int VEC>
__device__ __forceinline__ Pair thread_sum(const Weights& w, int lead, int lo, int hi, int lane)
{
    Sum2 sum;
    Pair rest = {0.f, 0.f};
    auto careful = [&](int i, float x, float y) { rest = add(rest, w.one(i, x, y)); };
    if (VEC == 1 || w.ngone > 0) {
        for_slice<BF16, VEC>(
            w.p, w.q, lead, lo, hi, lane,
            [&](int i, const float (&x)[VEC], const float (&y)[VEC]) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) careful(i + k, x[k], y[k]);
            },
            careful);
        return rest;
    }
    // negative entries and NaN become zero on the way; for an infinite one, which
    // shows in the sum or in q's largest, the thread goes over its entries again
    float top = 0.f;
    for_slice<BF16, VEC>(
        w.p, w.q, lead, lo, hi, lane,
        [&](int, const float (&x)[VEC], const float (&y)[VEC]) {
#pragma unroll
            for (int k = 0; k + 1 < VEC; k += 2) {
                if (w.q) {
                    top = fmaxf(top, fmaxf(y[k], y[k + 1]));
                    w.two(pack2(x[k], x[k + 1]), pack2(fmaxf(y[k], 0.f), fmaxf(y[k + 1], 0.f)), sum);
                } else {
                    sum.add(pack2(fmaxf(x[k], 0.f), fmaxf(x[k + 1], 0.f)));
                }
            }
        },
        careful);
    const Pair fast = sum.value();
    if (top < INFINITY && fast.hi < INFINITY) return add(fast, rest);
    rest = {0.f, 0.f};
    for_slice<BF16, VEC>(
        w.p, w.q, lead, lo, hi, lane,
        [&](int i, const float (&x)[VEC], const float (&y)[VEC]) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) careful(i + k, x[k], y[k]);
        },
        careful);
    return rest;
}

template <bool BF16, int VEC>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv_tree_verify_kernel(const VerifyParams prm)
{
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int s = blockIdx.x / ranks;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int ES = BF16 ? 2 : 4;
    // (the next kernel may start now, not before: all that was launched earlier is done)
    pdl_wait();
    pdl_launch_dependents();

    // ---- the tree, and the single probabilities at its tokens
    if (tid == 0) {
        int t0, n, bad = 0;
        if (!tree_span(prm.starts, s, prm.total, prm.max_nodes, t0, n, bad) && rank == 0)
            raise_flag(&g_verify_err, KV_DEVERR_BAD_TREE, bad);
        sh.t0 = t0;
        sh.n = n;
        sh.v = 0;
        sh.depth = 1;
        sh.ngone = 0;
        sh.a = {0.f, 0.f};
        sh.Z = {1.f, 0.f};
        sh.path[0] = 0;
    }
    __syncthreads();
    const int n = sh.n, t0 = sh.t0;
    if (n == 0) {                        // the whole cluster leaves together
        if (rank == 0) {
            if (tid == 0) prm.lens[s] = 0;
            for (int i = tid; i < prm.max_nodes; i += kThreads) {
                prm.nodes[(size_t)s * prm.max_nodes + i] = -1;
                prm.out[(size_t)s * prm.max_nodes + i] = -1;
            }
        }
        return;
    }
    // no CTA writes to another's shared memory before that one has started
    cg::cluster_group::arrival_token started = cluster.barrier_arrive();
    if (tid < n) {
        const int p = tree_parent(prm.parents, t0, tid, rank == 0 ? &g_verify_err : nullptr);
        const int x = __ldg(prm.tokens + t0 + tid);
        sh.par[tid] = p;
        sh.tok[tid] = x;
        bool takes = false;
        if (!prm.greedy && p >= 0 && x >= 0 && x < prm.vocab) {
            const long long prow = t0 + p;
            const float pv = clean(load1<BF16>(prm.target, prow * prm.target_stride + x));
            const float qv = prm.draft ? clean(load1<BF16>(prm.draft, prow * prm.draft_stride + x)) : 1.f;
            const float u = __ldg(prm.accept_u + t0 + tid);
            sh.pv[tid] = pv;
            sh.qv[tid] = qv;
            sh.u[tid] = u;
            takes = above(Pair{pv, 0.f}, mul(Pair{u, 0.f}, qv));
        }
        sh.takes[tid] = takes;
    }
    __syncthreads();
    if (tid < n) {
        int child = -1, sib = -1;
        const int mine = sh.par[tid];
#pragma unroll 4
        for (int j = n - 1; j > tid; --j) {
            const int p = sh.par[j];
            if (p == tid) child = j;
            if (p >= 0 && p == mine) sib = j;
        }
        sh.child[tid] = child;
        sh.sibling[tid] = sib;
    }
    __syncthreads();
    if (tid == 0) sh.next_child = sh.child[0];
    cluster.barrier_wait(std::move(started));

    int phase = 0;                       // which buffer the next exchange uses
    while (true) {
        __syncthreads();
        // ---- one thread walks until a row has to be read
        if (tid == 0) {
            int state = prm.greedy ? kNeedSum : kWalk;
            while (state == kWalk) {
                const int c = sh.next_child;
                if (c < 0) {
                    state = kDone;
                    break;
                }
                const int x = sh.tok[c];
                if (x < 0 || x >= prm.vocab) {
                    sh.next_child = sh.sibling[c];
                    continue;
                }
                bool takes = sh.takes[c];        // (as a first child)
                const bool refused = prm.draft ? sh.a.hi > 0.f : sh.ngone > 0;
                Pair r = {sh.pv[c], 0.f};
                if (refused) {
                    if (prm.draft) {
                        const Pair aq = mul(sh.a, sh.qv[c]);
                        r = add(r, Pair{-aq.hi, -aq.lo});
                    }
                    for (int g = 0; g < sh.ngone; ++g)
                        if (sh.gone[g] == x) r = {0.f, 0.f};
                    takes = r.hi > 0.f && above(r, mul(mul(Pair{sh.u[c], 0.f}, sh.qv[c]), sh.Z));
                }
                if (takes) {
                    sh.v = c;
                    sh.path[sh.depth++] = c;
                    sh.next_child = sh.child[c];
                    sh.a = {0.f, 0.f};
                    sh.Z = {1.f, 0.f};
                    sh.ngone = 0;
                } else {
                    sh.next_child = sh.sibling[c];
                    if (prm.draft) {
                        sh.a = add(sh.a, sh.Z);
                        // the last child's refusal is summed by the final pass
                        if (sh.next_child >= 0) state = kNeedSum;
                    } else {
                        sh.Z = add(sh.Z, Pair{-r.hi, -r.lo});
                        sh.gone[sh.ngone++] = x;
                    }
                }
            }
            sh.state = state;
        }
        __syncthreads();
        const int state = sh.state, v = sh.v;
        // ---- one pass over the node's rows
        const void* p = (const uint8_t*)prm.target + (long long)(t0 + v) * prm.target_stride * ES;
        const int lead = VEC > 1 ? (int)(((16 - ((uintptr_t)p & 15)) & 15) / ES) : 0;
        int lo, hi;
        warp_slice(prm.vocab, lead, VEC, rank * kWarps + warp, ranks * kWarps, lo, hi);

        if (prm.greedy) {
            float m = -INFINITY;
            int at = INT32_MAX;
            auto one = [&](int i, float x, float) {
                if (x > m) { m = x; at = i; }
            };
            for_slice<BF16, VEC>(p, nullptr, lead, lo, hi, lane,
                                 [&](int i, const float (&x)[VEC], const float (&)[VEC]) {
#pragma unroll
                                     for (int k = 0; k < VEC; ++k) one(i + k, x[k], 0.f);
                                 },
                                 one);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float om = __shfl_xor_sync(kFull, m, o);
                const int oa = __shfl_xor_sync(kFull, at, o);
                if (om > m || (om == m && oa < at)) { m = om; at = oa; }
            }
            if (lane == 0) { sh.wbest[warp] = m; sh.wbest_at[warp] = at; }
            __syncthreads();
            auto join = [&](int width) {     // over the first `width` lanes of a warp
                for (int o = width / 2; o > 0; o >>= 1) {
                    const float om = __shfl_xor_sync(kFull, m, o);
                    const int oa = __shfl_xor_sync(kFull, at, o);
                    if (om > m || (om == m && oa < at)) { m = om; at = oa; }
                }
            };
            if (warp == 0) {
                m = sh.wbest[lane & (kWarps - 1)];
                at = sh.wbest_at[lane & (kWarps - 1)];
                join(kWarps);
                if (lane < ranks) {
                    Shared* other = cluster.map_shared_rank(&sh, lane);
                    other->best[phase][rank] = m;
                    other->best_at[phase][rank] = at;
                }
            }
            cluster.sync();
            if (warp == 0) {
                m = -INFINITY;
                at = INT32_MAX;
                if (lane < ranks) {
                    m = sh.best[phase][lane];
                    at = sh.best_at[phase][lane];
                }
                join(kMaxCluster);
                if (lane == 0) {
                    if (at == INT32_MAX) at = 0;         // nothing but -inf and NaN
                    int c = sh.next_child;
                    while (c >= 0 && sh.tok[c] != at) c = sh.sibling[c];
                    if (c >= 0) {
                        sh.v = c;
                        sh.path[sh.depth++] = c;
                        sh.next_child = sh.child[c];
                    }
                    sh.state = c >= 0 ? kWalk : kDone;
                    sh.token = at;
                }
            }
            phase ^= 1;
            __syncthreads();
            if (sh.state == kDone) break;
            continue;
        }

        Weights w;
        const Pair a = sh.a;
        w.p = p;
        w.q = prm.draft && a.hi > 0.f
                  ? (const uint8_t*)prm.draft + (long long)(t0 + v) * prm.draft_stride * ES
                  : nullptr;
        w.ah = a.hi;
        w.al = a.lo;
        w.gone = sh.gone;
        w.ngone = prm.draft ? 0 : sh.ngone;
        // every warp's sum goes to every CTA
        const Pair ws = warp_sum(thread_sum<BF16, VEC>(w, lead, lo, hi, lane));
        if (lane < ranks) cluster.map_shared_rank(&sh, lane)->sums[phase][rank * kWarps + warp] = ws;
        cluster.sync();
        // the sums up to each warp: four consecutive warps a lane
        constexpr int kPer = kMaxCluster * kWarps / 32;
        Pair part[kPer], upto = {0.f, 0.f};
        const Pair* sums = sh.sums[phase];
        phase ^= 1;
        if (state == kNeedSum && warp != 0) continue;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = lane * kPer + k;
            part[k] = i < ranks * kWarps ? sums[i] : Pair{0.f, 0.f};
            upto = add(upto, part[k]);
        }
        const bool any = upto.hi > 0.f;
        upto = warp_scan(upto, lane);
        const Pair total = shfl(upto, 31);
        if (state == kNeedSum) {
            if (tid == 0) sh.Z = total;
            continue;
        }
        if (!(total.hi > 0.f) && (a.hi > 0.f || w.ngone > 0)) {
            // nothing is left of the target once the refused children are out:
            // the token comes from the target itself
            if (tid == 0) {
                sh.a = {0.f, 0.f};
                sh.ngone = 0;
            }
            continue;
        }
        // ---- the first entry whose cumulative sum is above t = u * total: the warp of
        // the cluster whose slice holds it; then that CTA's warps, in equal shares of
        // the slice, look for it, and the lanes of the one that has it
        const Pair t = mul(total, fmaxf(__ldg(prm.sample_u + s), 0.f));
        const unsigned some = __ballot_sync(kFull, any);
        if (some == 0) {                 // no weight at all
            if (rank != 0) return;
            if (tid == 0) sh.token = -1;
            __syncthreads();
            break;
        }
        const unsigned over = __ballot_sync(kFull, above(upto, t));
        // (u >= 1, or rounding: the last warp with any weight)
        const int src = over ? __ffs(over) - 1 : 31 - __clz(some);
        Pair run = shfl(upto, src > 0 ? src - 1 : 0);
        if (src == 0) run = {0.f, 0.f};
        int ow = -1;
        {
            int pick = -1, last = 0;
            Pair c = run, b = run, lb = run;
            if (lane == src) {
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    const Pair up = add(c, part[k]);
                    if (part[k].hi > 0.f) {
                        last = k;
                        lb = c;
                    }
                    if (pick < 0 && above(up, t)) {
                        pick = k;
                        b = c;
                    }
                    c = up;
                }
                if (pick < 0) {
                    pick = last;
                    b = lb;
                }
            }
            ow = src * kPer + __shfl_sync(kFull, pick, src);
            run = shfl(b, src);
        }
        if (rank != ow / kWarps) return;
        warp_slice(prm.vocab, lead, VEC, ow, ranks * kWarps, lo, hi);
        // a share's sum, lanes side by side
        const int per = (hi - lo + kWarps - 1) / kWarps;
        int from = lo + warp * per, end = min(from + per, hi);
        Pair sum = {0.f, 0.f};
#pragma unroll 4
        for (int i = from + lane; i < end; i += 32)
            sum = add(sum, w.one(i, load1<BF16>(w.p, i), w.q ? load1<BF16>(w.q, i) : 0.f));
        sum = warp_sum(sum);
        Pair* shares = sh.sums[phase];           // (the exchange after next is not to come)
        if (lane == 0) shares[warp] = sum;
        __syncthreads();
        // Of consecutive shares, one a lane with its sum: the one that holds the cut, and
        // the sum up to it.  (Rounding may leave none above t: the last with any weight.)
        auto cut = [&](Pair mine, Pair& upto_it) -> int {
            const Pair incl = add(upto_it, warp_scan(mine, lane));
            const unsigned hit = __ballot_sync(kFull, above(incl, t));
            const unsigned pos = __ballot_sync(kFull, mine.hi > 0.f);
            const int l = hit ? __ffs(hit) - 1 : pos ? 31 - __clz(pos) : 0;
            const Pair before = shfl(incl, l > 0 ? l - 1 : 0);
            if (l > 0) upto_it = before;
            return l;
        };
        const int share = cut(lane < kWarps ? shares[lane] : Pair{0.f, 0.f}, run);
        if (warp == min(share, kWarps - 1)) {
            // the warp's entries in equal consecutive shares of the lanes, until a share
            // is one entry
            int cnt = end - from;
            while (true) {
                const int each = (cnt + 31) / 32, i0 = from + lane * each, i1 = min(i0 + each, from + cnt);
                Pair x = {0.f, 0.f};
#pragma unroll 4
                for (int i = i0; i < i1; ++i)
                    x = add(x, w.one(i, load1<BF16>(w.p, i), w.q ? load1<BF16>(w.q, i) : 0.f));
                const int l = cut(x, run);
                from += l * each;
                cnt = min(each, cnt - l * each);
                if (each <= 1) break;
            }
            if (lane == 0) sh.token = min(from, prm.vocab - 1);
        }
        __syncthreads();
        break;
    }
    // ---- results, from the one CTA that is left (greedy: the first)
    if (prm.greedy && rank != 0) return;
    const int depth = sh.depth, token = sh.token;
    if (tid == 0) prm.lens[s] = depth;
    for (int i = tid; i < prm.max_nodes; i += kThreads) {
        const size_t at = (size_t)s * prm.max_nodes + i;
        prm.nodes[at] = i < depth ? sh.path[i] : -1;
        prm.out[at] = i + 1 < depth ? sh.tok[sh.path[i + 1]] : (i + 1 == depth ? token : -1);
    }
}

template <bool BF16, int VEC>
cudaError_t launch_verify(const VerifyParams& p, int num_seqs, int cluster, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_seqs * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kv_tree_verify_kernel<BF16, VEC>, p);
}

}  // namespace

int verify_read_error(unsigned* flags, long long* detail) { return g_launched.take_error(g_verify_err, flags, detail); }

}  // namespace pkv

using namespace pkv;

extern "C" int kv_tree_verify(int32_t* accept_lens, int32_t* accept_nodes, int32_t* out_tokens,
                              const void* target_probs, int64_t target_stride,
                              const void* draft_probs, int64_t draft_stride, int prob_dtype,
                              const int32_t* tokens, const int32_t* parents,
                              const int32_t* node_starts, const float* accept_u,
                              const float* sample_u, int num_seqs, int total_nodes, int max_nodes,
                              int vocab, unsigned flags, void* stream)
{
    if (num_seqs < 0 || total_nodes < 0 || max_nodes < 1 || vocab < 1) return KV_ERR_INVALID_ARG;
    if (max_nodes > KV_TREE_MAX_NODES) return KV_ERR_TOO_LARGE;
    if (flags & ~KV_VERIFY_GREEDY) return KV_ERR_INVALID_ARG;
    if (prob_dtype != KV_DTYPE_F32 && prob_dtype != KV_DTYPE_BF16) return KV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return KV_OK;
    const bool greedy = flags & KV_VERIFY_GREEDY, bf16 = prob_dtype == KV_DTYPE_BF16;
    if (!accept_lens || !accept_nodes || !out_tokens || !node_starts) return KV_ERR_INVALID_ARG;
    if (total_nodes > 0 && (!target_probs || !tokens || (!greedy && (!accept_u || !sample_u))))
        return KV_ERR_INVALID_ARG;
    if (greedy) draft_probs = nullptr;
    if (target_stride < vocab || (draft_probs && draft_stride < vocab)) return KV_ERR_INVALID_ARG;
    const uintptr_t es = bf16 ? 2 : 4;
    if (((uintptr_t)target_probs | (uintptr_t)draft_probs) % es != 0) return KV_ERR_INVALID_ARG;
    if (vocab > INT32_MAX / 2) return KV_ERR_UNSUPPORTED;
    VerifyParams p;
    p.lens = accept_lens;
    p.nodes = accept_nodes;
    p.out = out_tokens;
    p.target = target_probs;
    p.draft = draft_probs;
    p.target_stride = target_stride;
    p.draft_stride = draft_stride;
    p.tokens = tokens;
    p.parents = parents;
    p.starts = node_starts;
    p.accept_u = accept_u;
    p.sample_u = sample_u;
    p.total = total_nodes;
    p.max_nodes = max_nodes;
    p.vocab = vocab;
    p.greedy = greedy;
    // 16-byte loads where the two rows of every node are aligned alike
    const bool vec = !draft_probs ||
                     (((uintptr_t)target_probs - (uintptr_t)draft_probs) % 16 == 0 &&
                      (target_stride - draft_stride) * (int64_t)es % 16 == 0);
    // all sequences at once, where they fit: a second wave would wait for the first
    // one's walks (64 trees, 128000 entries: 139 us with clusters of 8)
    int cluster = kMaxCluster;
    while (cluster > 1 && (long long)num_seqs * cluster > kCtasPerSm * num_sms_current()) cluster /= 2;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    g_launched.note();
    const cudaError_t err =
        bf16 ? (vec ? launch_verify<true, 8>(p, num_seqs, cluster, st)
                    : launch_verify<true, 1>(p, num_seqs, cluster, st))
             : (vec ? launch_verify<false, 4>(p, num_seqs, cluster, st)
                    : launch_verify<false, 1>(p, num_seqs, cluster, st));
    return err == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}
