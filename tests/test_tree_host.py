"""Host side of decoding with drafted trees, on the CPU: reserving places for a
tree (kv_tree_step), cutting a sequence back (kv_seq_truncate), what the entry
points refuse, and the verification rule itself (the 64-bit reference's emitted
tokens follow the target's distribution)."""
import ctypes

import numpy as np
import pytest
import torch

import tree_reference as R


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build_native()
    import paged_kv_cache_21_gb300 as pk
    return pk


def test_one_node_is_kv_step(pk):
    a, b = pk.BlockAllocator(64, 2, 64), pk.BlockAllocator(64, 2, 64)
    for x in (a, b):
        x.add(7, 0)
        x.add(8, 16)
        x.add(9, 21)
        x.fork(9, 10, 20)
    for _ in range(20):
        sa, ta, la, ca = a.step([7, 8, 9, 10], 8)
        sb, tb, lb, starts, cb = b.tree_step([7, 8, 9, 10], [1, 1, 1, 1], 8)
        assert np.array_equal(sa, sb) and np.array_equal(ta, tb) and np.array_equal(la, lb)
        assert np.array_equal(starts, np.arange(5))
        assert np.array_equal(ca[0], cb[0]) and np.array_equal(ca[1], cb[1])


def test_slots_follow_the_block_table_and_truncate_returns_blocks(pk):
    rng = np.random.default_rng(0)
    a = pk.BlockAllocator(200, 2, 64)
    lens = {}
    for i in range(6):
        lens[i] = int(rng.integers(0, 60))
        a.add(i, lens[i])
    for _ in range(60):
        counts = rng.integers(0, 40, size=6)
        slots, bt, cl, starts, cow = a.tree_step(list(range(6)), counts, 12)
        assert starts[0] == 0 and np.array_equal(np.diff(starts), counts)
        for s in range(6):
            assert cl[s] == lens[s] + counts[s]
            pos = np.arange(lens[s], cl[s])
            assert np.array_equal(slots[starts[s]:starts[s + 1]],
                                  bt[s, pos // 16].astype(np.int64) * 16 + pos % 16)
        held = bt[bt >= 0]
        assert len(set(held.tolist())) == len(held)              # nothing is shared here
        keep = [int(rng.integers(lens[s], cl[s] + 1)) if lens[s] < 100 else lens[s] // 3
                for s in range(6)]
        a.truncate(list(range(6)), keep)
        lens = dict(enumerate(keep))
        need = sum(-(-x // 16) for x in keep)
        assert a.stats()[:2] == (200 - need, need)
        assert [r["len"] for r in a.trace(list(range(6)))] == keep


def test_a_shared_tail_is_copied_and_a_shared_block_survives_truncation(pk):
    a = pk.BlockAllocator(20, 1, 64)
    a.add(0, 20)                                   # blocks 0, 1 (1 partial)
    a.fork(0, 1, 20)
    a.fork(0, 2, 16)                               # shares block 0 only
    slots, bt, cl, starts, (src, dst) = a.tree_step([0, 1, 2], [5, 30, 2], 8)
    assert len(src) == 1 and src[0] == 1           # the first copies, the second owns it then
    assert bt[0, 1] == dst[0] and bt[1, 1] == 1
    assert a.stats(0)[3] == 3
    a.truncate([1, 2], [3, 0])
    assert a.stats(0)[3] == 2                      # 0 and 1 still hold block 0
    assert a.stats(1)[3] == 0
    assert a.info(2)[0] == 0 and len(a.info(2)[1]) == 0


def test_tree_step_is_all_or_nothing(pk):
    a = pk.BlockAllocator(4, 1, 64)
    a.add(0, 17)
    a.add(1, 3)
    before = (a.trace(), a.stats())
    bad = [([0, 1], [40, 40], 8, pk.KV_ERR_OUT_OF_BLOCKS),
           ([0, 5], [1, 1], 8, pk.KV_ERR_NOT_FOUND),
           ([0, 0], [1, 1], 8, pk.KV_ERR_INVALID_ARG),
           ([0, 1], [1, -1], 8, pk.KV_ERR_INVALID_ARG),
           ([0, 1], [16, 1], 2, pk.KV_ERR_INVALID_ARG)]
    for ids, counts, mb, code in bad:
        with pytest.raises(pk.KVError) as e:
            a.tree_step(ids, counts, mb)
        assert e.value.code == code
    a.fork(1, 2, 3)
    with pytest.raises(pk.KVError) as e:           # the copy-on-write pair has no room
        a.tree_step([1], [2], 8, cow_cap=0)
    assert e.value.code == pk.KV_ERR_INVALID_ARG
    a.free(2)
    assert (a.trace(), a.stats()) == before
    for ids, lens, code in [([0], [18], pk.KV_ERR_INVALID_ARG), ([0], [-1], pk.KV_ERR_INVALID_ARG),
                            ([0, 9], [1, 1], pk.KV_ERR_NOT_FOUND),
                            ([1, 1], [1, 1], pk.KV_ERR_INVALID_ARG)]:
        with pytest.raises(pk.KVError) as e:
            a.truncate(ids, lens)
        assert e.value.code == code
    assert (a.trace(), a.stats()) == before
    L = pk._lib
    assert L.kv_tree_step(None, None, None, 0, None, None, 1, None, None, None, None, 0,
                          None) == pk.KV_ERR_INVALID_ARG
    assert L.kv_seq_truncate(a._h, None, None, 1) == pk.KV_ERR_INVALID_ARG
    slots, bt, cl, starts, _ = a.tree_step([], [], 4)
    assert len(slots) == 0 and list(starts) == [0]


def test_entry_points_refuse_bad_arguments_before_any_launch(pk):
    """Through the C ABI, with addresses that are never read."""
    L, X = pk._lib, ctypes.c_void_p(4096)
    ok = dict(out=X, odt=0, q=X, k=X, v=X, dt=0, ks=1.0, vs=1.0, nb=8, bt=X, mb=4, cl=X, st=X,
              par=X, B=2, T=6, mx=4, hq=8, hkv=2, d=64, scale=0.1, ws=X, wb=1 << 40, stream=None)

    def attend(**kw):
        a = dict(ok, **kw)
        return L.paged_tree_attention(*a.values())

    E, U, T = pk.KV_ERR_INVALID_ARG, pk.KV_ERR_UNSUPPORTED, pk.KV_ERR_TOO_LARGE
    odd = ctypes.c_void_p(4100)
    for kw, code in [(dict(B=-1), E), (dict(mx=0), E), (dict(mx=129), T), (dict(hq=7), E),
                     (dict(d=96), U), (dict(dt=2), U), (dict(odt=1), U), (dict(T=-1), E),
                     (dict(out=None), E), (dict(q=None), E), (dict(k=None), E), (dict(v=None), E),
                     (dict(bt=None), E), (dict(cl=None), E), (dict(st=None), E),
                     (dict(ws=None), E), (dict(nb=0), E), (dict(mb=0), E), (dict(q=odd), E),
                     (dict(out=odd), E), (dict(k=odd), E), (dict(scale=float("nan")), E),
                     (dict(dt=1, ks=0.0), E), (dict(dt=1, vs=float("inf")), E),
                     (dict(hq=260, hkv=2), U), (dict(B=0), 0), (dict(T=0), 0)]:
        assert attend(**kw) == code, kw

    okv = dict(al=X, an=X, ot=X, tp=X, ts=100, dp=X, ds=100, dt=2, tok=X, par=X, st=X, au=X, su=X,
               B=2, T=6, mx=4, V=100, fl=0, stream=None)

    def verify(**kw):
        return L.kv_tree_verify(*dict(okv, **kw).values())

    for kw, code in [(dict(B=-1), E), (dict(T=-1), E), (dict(mx=0), E), (dict(mx=129), T),
                     (dict(V=0), E), (dict(fl=2), E), (dict(dt=1), U), (dict(al=None), E),
                     (dict(an=None), E), (dict(ot=None), E), (dict(tp=None), E),
                     (dict(tok=None), E), (dict(st=None), E), (dict(au=None), E),
                     (dict(su=None), E), (dict(ts=99), E), (dict(ds=99), E),
                     (dict(tp=ctypes.c_void_p(4098)), E), (dict(B=0), 0)]:
        assert verify(**kw) == code, kw

    ptrs = (ctypes.c_void_p * 2)(4096, 8192)
    bad = (ctypes.c_void_p * 2)(4096, 0)
    okc = dict(k=ptrs, v=ptrs, nl=2, bt=X, mb=4, cl=X, st=X, an=X, al=X, B=2, mx=4, hkv=2, d=64,
               nb=8, dt=0, stream=None)

    def compact(**kw):
        return L.kv_tree_compact(*dict(okc, **kw).values())

    for kw, code in [(dict(nl=-1), E), (dict(B=-1), E), (dict(mx=0), E), (dict(mx=129), T),
                     (dict(hkv=0), E), (dict(d=0), E), (dict(d=12, dt=0), U), (dict(dt=2), U),
                     (dict(nb=0), E), (dict(mb=0), E), (dict(k=None), E), (dict(v=bad), E),
                     (dict(bt=None), E), (dict(cl=None), E), (dict(st=None), E),
                     (dict(an=None), E), (dict(al=None), E), (dict(B=0), 0), (dict(nl=0), 0)]:
        assert compact(**kw) == code, kw
    # caches that overlap: 8 blocks x 2 heads x 16 x 128 bytes = 32 KB each
    size = 8 * 2 * 16 * 128
    for v in ([1 << 20, (1 << 20) + 2 * size], [(1 << 20) + size - 16, 1 << 22], [4096, 4096]):
        assert compact(k=(ctypes.c_void_p * 2)(1 << 20, 1 << 21), v=(ctypes.c_void_p * 2)(*v)) == E


def test_the_binding_refuses_tensors_of_the_wrong_type_or_place(pk):
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    kc = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(1024, dtype=torch.uint8)
    good = [torch.empty_like(q), q, kc, kc, i32(1, 2), i32(1), i32(2), i32(3), 3, 0.1, ws]
    for at, what in [(0, torch.zeros((3, 4, 64), dtype=torch.float16)),
                     (0, torch.zeros((2, 4, 64), dtype=torch.bfloat16)), (1, q.float()),
                     (1, torch.zeros((4, 3, 64), dtype=torch.bfloat16).transpose(0, 1)),
                     (3, kc[:3]), (3, kc.to(torch.uint8))]:
        bad = list(good)
        bad[at] = what
        with pytest.raises(ValueError):
            pk.paged_tree_attention(*bad)
    with pytest.raises(ValueError, match="pinned"):        # plain host memory
        pk.paged_tree_attention(*good)
    with pytest.raises(ValueError):
        pk.CacheLayers([kc], [kc[:2]])
    with pytest.raises(ValueError):
        pk.CacheLayers([], [])
    P = torch.zeros((3, 10))
    args = [i32(1), i32(1, 3), i32(1, 3), P, i32(3), i32(3), i32(2), torch.zeros(3),
            torch.zeros(1)]
    for at, what in [(3, P.double()), (3, torch.zeros((10, 3)).t()), (7, None),
                     (7, torch.zeros(4)), (8, torch.zeros(1).double())]:
        bad = list(args)
        bad[at] = what
        with pytest.raises(ValueError):
            pk.kv_tree_verify(*bad)
    with pytest.raises(ValueError):
        pk.kv_tree_verify(*args, draft_probs=torch.zeros((3, 9)))


@pytest.mark.parametrize("kids,drawn", [(1, True), (3, True), (1, False), (3, False)])
def test_the_rule_emits_the_targets_distribution(kids, drawn):
    """First emitted token of 60000 one-level trees: with children drawn from q
    (or chosen, distinct), it is distributed as the target's p.  A share's
    standard deviation is sqrt(p (1 - p) / N) <= 0.5 / sqrt(N); 5 of them."""
    rng = np.random.default_rng(kids)
    V, N = 6, 60000
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    n = kids + 1
    par = np.array([-1] + [0] * kids)
    count = np.zeros(V)
    target, draft = np.tile(p, (n, 1)), np.tile(q, (n, 1))
    starts = np.array([0, n])
    for _ in range(N):
        toks = rng.choice(V, size=n, p=q) if drawn else np.array([0, 4, 1, 2])[:n]
        _, _, out = R.verify(target, draft if drawn else None, toks, par, starts, rng.random(n),
                             rng.random(1), n)
        count[out[0, 0]] += 1
    assert np.abs(count / N - p).max() < 5 * 0.5 / np.sqrt(N)
