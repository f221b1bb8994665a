// Draft-tree tables shared by the kernels that read them (paged_tree.cu,
// tree_verify.cu, kv_compact.cu), dependent launches, and arithmetic on two floats at
// a time.
#pragma once

#include "device_common.cuh"
#include "paged_kv.h"

namespace pkv {

// A kernel of a chain of dependent launches: wait until the kernels before it have
// completed; let the next one start.
__device__ __forceinline__ void pdl_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void pdl_launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

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

using u64 = unsigned long long;          // two floats, the first in the low half

__device__ __forceinline__ u64 pack2(float a, float b)
{
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(u64 x, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ u64 add2(u64 a, u64 b)
{
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 sub2(u64 a, u64 b)
{
    u64 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b)
{
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c)
{
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

}  // namespace pkv
