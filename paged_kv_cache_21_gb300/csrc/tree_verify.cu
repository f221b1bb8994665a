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
// entries' spacing in them: float32 would move one sampled token in a few
// dozen.  Each thread sums in pairs of floats (two-sum, 2^-48), which costs a
// tenth of the time of this GPU's double precision units; the few sums over
// threads run in double.
//
// One cluster of CTAs serves a sequence: each CTA takes a contiguous slice of
// the row, its warps contiguous sub-slices, and the CTAs exchange their sums
// through distributed shared memory.  All CTAs walk the tree in step, from
// copies of the tree and of the single probabilities at the drafted tokens
// (gathered at once, for all nodes) in shared memory.  The CTA, warp and lane
// that hold the cut then find the token; the row comes from L2 by then.
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

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
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

// A float32 sum carried with its rounding error.
struct Sum2 {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x, float xe)
    {
        const float s = hi + x, b = s - hi;
        lo += ((hi - (s - b)) + (x - b)) + xe;
        hi = s;
    }
    __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

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

// The remaining weight of an entry as a float and its error: max(p - a q, 0)
// with a = ah + al, the product and the difference exact but for 2^-48.
struct Residual {
    float ah = 0.f, al = 0.f;            // refusals so far; 0: the target itself
    __device__ __forceinline__ float2 operator()(float p, float q) const
    {
        const float ph = __fmul_rn(ah, q);   // not to be contracted into the difference
        const float pe = fmaf(ah, q, -ph) + al * q;
        const float s = p - ph, b = s - p;
        const float e = ((p - (s - b)) + (-ph - b)) - pe;
        return s + e > 0.f ? make_float2(s, e) : make_float2(0.f, 0.f);
    }
};

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Shared state of a CTA.  Every CTA of a cluster holds the same tree and walk.
struct Shared {
    int tok[kN], child[kN], sibling[kN];     // first child and next sibling, -1: none
    float pv[kN], qv[kN], u[kN];             // p and q of the node's token at its parent
    int gone[kN];                            // refused tokens of the node (no draft)
    int path[kN];
    double warp_sums[kWarps];
    double rank_sums[2][kMaxCluster];
    float best[2][kMaxCluster];              // greedy: largest entry and where it is
    int best_at[2][kMaxCluster];
    float wbest[kWarps];
    int wbest_at[kWarps];
    double a, Z;
    int v, next_child, ngone, depth, state, n, t0;
};

enum State { kWalk, kNeedSum, kDone };

// The rows of one node, cut into aligned vectors: entry 0 is element `shift`
// of its first vector.
template <bool BF16, int VEC>
struct Rows {
    const void* p;
    const void* q;
    int vocab;
    int lead;                                // entries before the first whole vector

    template <typename F>
    __device__ __forceinline__ void for_each(int lo, int hi, int lane, F&& f) const
    {
        // entries lo .. hi of the row; lo is lead + a multiple of 32 * VEC, or 0
        int i = lo;
        if (VEC > 1 && lo == 0 && lead > 0) {
            if (lane < lead && lane < hi) {
                float x[1] = {load1<BF16>(p, lane)}, y[1] = {q ? load1<BF16>(q, lane) : 0.f};
                f(lane, 1, x, y);
            }
            i = lead;
        }
#pragma unroll 4
        for (int at = i + lane * VEC; at + VEC <= hi; at += 32 * VEC) {
            float x[VEC], y[VEC];
            loadv<BF16, VEC>(p, at, x);
            if (q) {
                loadv<BF16, VEC>(q, at, y);
            } else {
#pragma unroll
                for (int k = 0; k < VEC; ++k) y[k] = 0.f;
            }
            f(at, VEC, x, y);
        }
        if (VEC > 1 && hi > i) {
            const int tail = (hi - i) % VEC, at = hi - tail + lane;
            if (lane < tail) {
                float x[1] = {load1<BF16>(p, at)}, y[1] = {q ? load1<BF16>(q, at) : 0.f};
                f(at, 1, x, y);
            }
        }
    }
};

// The slice [lo, hi) of warp `w` of `nw` over the whole cluster.
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

template <bool BF16, int VEC>
__global__ void __launch_bounds__(kThreads) kv_tree_verify_kernel(const VerifyParams prm)
{
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int s = blockIdx.x / ranks;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int ES = BF16 ? 2 : 4;

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
        sh.a = 0.0;
        sh.Z = 1.0;
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
    __shared__ int par[kN];
    if (tid < n) {
        const int p = tree_parent(prm.parents, t0, tid, rank == 0 ? &g_verify_err : nullptr);
        par[tid] = p;
        const int x = __ldg(prm.tokens + t0 + tid);
        sh.tok[tid] = x;
        sh.pv[tid] = 0.f;
        if (!prm.greedy && p >= 0 && x >= 0 && x < prm.vocab) {
            const long long prow = t0 + p;
            sh.pv[tid] = clean(load1<BF16>(prm.target, prow * prm.target_stride + x));
            sh.qv[tid] = prm.draft ? clean(load1<BF16>(prm.draft, prow * prm.draft_stride + x)) : 1.f;
            sh.u[tid] = __ldg(prm.accept_u + t0 + tid);
        }
    }
    __syncthreads();
    if (tid < n) {
        int child = -1, sib = -1;
        for (int j = n - 1; j > tid; --j) {
            const int p = par[j];
            if (p == tid) child = j;
            if (p >= 0 && p == par[tid]) sib = j;
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
                const double p = sh.pv[c], q = sh.qv[c];
                double r = p - sh.a * q;
                if (!prm.draft) {
                    r = p;
                    for (int g = 0; g < sh.ngone; ++g)
                        if (sh.gone[g] == x) r = 0.0;
                }
                if (r < 0.0) r = 0.0;
                if ((double)sh.u[c] * q * sh.Z < r) {
                    sh.v = c;
                    sh.path[sh.depth++] = c;
                    sh.next_child = sh.child[c];
                    sh.a = 0.0;
                    sh.Z = 1.0;
                    sh.ngone = 0;
                } else {
                    sh.next_child = sh.sibling[c];
                    if (prm.draft) {
                        sh.a += sh.Z;
                        // the last child's refusal is summed by the final pass
                        if (sh.next_child >= 0) state = kNeedSum;
                    } else {
                        sh.Z -= r;
                        sh.gone[sh.ngone++] = x;
                    }
                }
            }
            sh.state = state;
        }
        __syncthreads();
        const int state = sh.state;
        const int v = sh.v;
        // ---- one pass over the node's rows
        Rows<BF16, VEC> rows;
        rows.p = (const uint8_t*)prm.target + (long long)(t0 + v) * prm.target_stride * ES;
        Residual res;
        const double a = sh.a;
        res.ah = (float)a;
        res.al = (float)(a - (double)res.ah);
        rows.q = prm.draft && a > 0.0
                     ? (const uint8_t*)prm.draft + (long long)(t0 + v) * prm.draft_stride * ES
                     : nullptr;
        rows.vocab = prm.vocab;
        rows.lead = VEC > 1 ? (int)(((16 - ((uintptr_t)rows.p & 15)) & 15) / ES) : 0;
        int lo, hi;
        warp_slice(prm.vocab, rows.lead, VEC, rank * kWarps + warp, ranks * kWarps, lo, hi);

        if (prm.greedy) {
            float m = -INFINITY;
            int at = INT32_MAX;
            rows.for_each(lo, hi, lane, [&](int i, int cnt, const float* x, const float*) {
                for (int k = 0; k < cnt; ++k)
                    if (x[k] > m) { m = x[k]; at = i + k; }
            });
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float om = __shfl_xor_sync(kFull, m, o);
                const int oa = __shfl_xor_sync(kFull, at, o);
                if (om > m || (om == m && oa < at)) { m = om; at = oa; }
            }
            if (lane == 0) { sh.wbest[warp] = m; sh.wbest_at[warp] = at; }
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w < kWarps; ++w)
                    if (sh.wbest[w] > m || (sh.wbest[w] == m && sh.wbest_at[w] < at)) {
                        m = sh.wbest[w];
                        at = sh.wbest_at[w];
                    }
                for (int r = 0; r < ranks; ++r) {
                    Shared* other = cluster.map_shared_rank(&sh, r);
                    other->best[phase][rank] = m;
                    other->best_at[phase][rank] = at;
                }
            }
            cluster.sync();
            m = -INFINITY;
            at = INT32_MAX;
            for (int r = 0; r < ranks; ++r)
                if (sh.best[phase][r] > m || (sh.best[phase][r] == m && sh.best_at[phase][r] < at)) {
                    m = sh.best[phase][r];
                    at = sh.best_at[phase][r];
                }
            if (at == INT32_MAX) at = 0;         // nothing but -inf and NaN
            phase ^= 1;
            if (tid == 0) {
                int c = sh.next_child;
                while (c >= 0 && sh.tok[c] != at) c = sh.sibling[c];
                if (c >= 0) {
                    sh.v = c;
                    sh.path[sh.depth++] = c;
                    sh.next_child = sh.child[c];
                }
                sh.state = c >= 0 ? kWalk : kDone;
            }
            __syncthreads();
            if (sh.state == kDone) {
                if (tid == 0 && rank == 0) sh.gone[0] = at;
                __syncthreads();
                break;
            }
            continue;
        }

        const int ngone = prm.draft ? 0 : sh.ngone;
        auto weight = [&](int i, float x, float y) -> float2 {
            float w = clean(x);
            for (int g = 0; g < ngone; ++g)
                if (sh.gone[g] == i) w = 0.f;
            return res(w, clean(y));
        };
        Sum2 acc;
        rows.for_each(lo, hi, lane, [&](int i, int cnt, const float* x, const float* y) {
            for (int k = 0; k < cnt; ++k) {
                const float2 w = weight(i + k, x[k], y[k]);
                acc.add(w.x, w.y);
            }
        });
        const double wsum = warp_sum(acc.value());
        if (lane == 0) sh.warp_sums[warp] = wsum;
        __syncthreads();
        if (tid == 0) {
            double t = 0.0;
            for (int w = 0; w < kWarps; ++w) t += sh.warp_sums[w];
            for (int r = 0; r < ranks; ++r)
                cluster.map_shared_rank(&sh, r)->rank_sums[phase][rank] = t;
        }
        cluster.sync();
        double total = 0.0;
        for (int r = 0; r < ranks; ++r) total += sh.rank_sums[phase][r];
        if (state == kNeedSum) {
            if (tid == 0) sh.Z = total;
            phase ^= 1;
            continue;
        }
        if (total <= 0.0 && (a > 0.0 || ngone > 0)) {
            // nothing is left of the target once the refused children are out:
            // the token comes from the target itself
            if (tid == 0) {
                sh.a = 0.0;
                sh.ngone = 0;
            }
            phase ^= 1;
            continue;
        }
        // ---- the first entry whose cumulative sum is above u * total
        const double t = (double)__ldg(prm.sample_u + s) * total;
        double before = 0.0;
        int owner = -1, last = -1;
        double owner_before = 0.0, last_before = 0.0;
        for (int r = 0; r < ranks; ++r) {
            const double x = sh.rank_sums[phase][r];
            if (x > 0.0) {
                last = r;
                last_before = before;
            }
            if (owner < 0 && before + x > t) {
                owner = r;
                owner_before = before;
            }
            before += x;
        }
        if (owner < 0) {                 // u >= 1 or rounding: the last entry there is
            owner = last;
            owner_before = last_before;
        }
        if (owner < 0) {                 // no weight at all
            if (tid == 0) sh.gone[0] = -1;
            if (rank != 0) return;
            __syncthreads();
            break;
        }
        if (rank != owner) return;
        // the warp, then the 32 * VEC entries, then the entry
        int ow = -1, lw = -1;
        double b = owner_before, ow_before = 0.0, lw_before = 0.0;
        for (int w = 0; w < kWarps; ++w) {
            const double x = sh.warp_sums[w];
            if (x > 0.0) {
                lw = w;
                lw_before = b;
            }
            if (ow < 0 && b + x > t) {
                ow = w;
                ow_before = b;
            }
            b += x;
        }
        if (ow < 0) {
            ow = lw;
            ow_before = lw_before;
        }
        if (warp == ow) {
            double run = ow_before;
            int found = -1, last_pos = -1;
            for (int g0 = lo; g0 < hi && found < 0;) {
                // a group of entries in row order: the lead, whole vectors, or the tail
                const int first = VEC > 1 && g0 == 0 && rows.lead > 0 ? min(rows.lead, hi)
                                                                      : min(g0 + 32 * VEC, hi);
                const int cnt = first - g0;
                const int per = (cnt + 31) / 32;         // entries of a lane, in order
                double mine = 0.0;
                int lastk = -1;
                for (int k = 0; k < per; ++k) {
                    const int i = g0 + lane * per + k;
                    if (i < first) {
                        const float2 w = weight(i, load1<BF16>(rows.p, i),
                                                rows.q ? load1<BF16>(rows.q, i) : 0.f);
                        mine += (double)w.x + (double)w.y;
                        if (w.x > 0.f) lastk = i;
                    }
                }
                double incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double up = __shfl_up_sync(kFull, incl, o);
                    if (lane >= o) incl += up;
                }
                const unsigned hit = __ballot_sync(kFull, run + incl > t);
                if (hit) {
                    const int src = __ffs(hit) - 1;
                    if (lane == src) {
                        double c = run + (incl - mine);
                        for (int k = 0; k < per; ++k) {
                            const int i = g0 + lane * per + k;
                            if (i >= first) break;
                            const float2 w = weight(i, load1<BF16>(rows.p, i),
                                                    rows.q ? load1<BF16>(rows.q, i) : 0.f);
                            c += (double)w.x + (double)w.y;
                            if (c > t) {
                                found = i;
                                break;
                            }
                        }
                        if (found < 0) found = lastk;    // rounding: the lane's last entry
                    }
                    found = __shfl_sync(kFull, found, src);
                }
                const int lp = __reduce_max_sync(kFull, lastk);
                if (lp >= 0) last_pos = lp;
                run += __shfl_sync(kFull, incl, 31);
                g0 = first;
            }
            if (found < 0) found = last_pos;
            if (lane == 0) sh.gone[0] = found;
        }
        __syncthreads();
        break;
    }
    // ---- results, from the one CTA that is left (greedy: the first)
    if (prm.greedy && rank != 0) return;
    const int depth = sh.depth, token = sh.gone[0];
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
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_tree_verify_kernel<BF16, VEC>, p);
}

}  // namespace

int verify_read_error(unsigned* flags, long long* detail)
{
    DevErr e;
    if (cudaMemcpyFromSymbol(&e, g_verify_err, sizeof e) != cudaSuccess) return KV_ERR_CUDA;
    DevErr z = {0u, -1LL};
    if (cudaMemcpyToSymbol(g_verify_err, &z, sizeof z) != cudaSuccess) return KV_ERR_CUDA;
    *flags = e.flags;
    *detail = e.flags ? e.detail : -1;
    return KV_OK;
}

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
    int cluster = kMaxCluster;
    while (cluster > 1 && (long long)num_seqs * cluster > INT32_MAX) cluster /= 2;
    if ((long long)num_seqs * cluster > INT32_MAX) return KV_ERR_TOO_LARGE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err =
        bf16 ? (vec ? launch_verify<true, 8>(p, num_seqs, cluster, st)
                    : launch_verify<true, 1>(p, num_seqs, cluster, st))
             : (vec ? launch_verify<false, 4>(p, num_seqs, cluster, st)
                    : launch_verify<false, 1>(p, num_seqs, cluster, st));
    return err == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}
