// Draft-tree tables shared by the kernels that read them (paged_tree.cu,
// tree_verify.cu, kv_compact.cu).
#pragma once

#include "device_common.cuh"
#include "paged_kv.h"

namespace pkv {

// First node and number of nodes of sequence s.  False, with no nodes and the
// bad value, for a pair of starts that breaks the rules.
__device__ __forceinline__ bool tree_span(const int32_t* __restrict__ starts, int s, int total,
                                          int max_nodes, int& t0, int& n, int& bad)
{
    const int a = __ldg(starts + s), b = __ldg(starts + s + 1);
    t0 = a;
    n = b - a;
    if (a >= 0 && b >= a && b <= total && n <= max_nodes) return true;
    bad = a < 0 || b < a ? a : b;
    t0 = 0;
    n = 0;
    return false;
}

// The parent of node i as the tables' rules read it: a value that breaks them
// is a root's (-1), and raises the flag if `e` is given.
__device__ __forceinline__ int tree_parent(const int32_t* __restrict__ parents, int t0, int i,
                                           DevErr* e)
{
    if (!parents) return i - 1;
    const int p = __ldg(parents + t0 + i);
    if (p >= KV_TREE_PAD && p < i) return p;
    if (e) raise_flag(e, KV_DEVERR_BAD_TREE, p);
    return -1;
}

}  // namespace pkv
