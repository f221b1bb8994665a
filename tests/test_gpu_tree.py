"""Decoding with trees of drafted tokens on the GPU: attention, verification and
compaction against the 64-bit reference, at the sizes, masks and values where
they can go wrong, and a run of all of them as a program uses them.

Attention tolerances.  The kernels accumulate scores in float32: a score's
error is at most D 2^-24 sum |q k| scale, for the values used here (normal,
scale 1/sqrt(D)) below 2^-13.  The weights are held with a relative error of
2^-16 (bf16 cache: bf16 high and low parts) or 2^-11 (E4M3 cache: f16).  An
output is a mean of visible V with those weights, so its error is below
(2^-13 + 2^-16 + ...) < 2^-12, or 2^-11 + 2^-12 < 2^-10, times twice the
largest |V| (numerator and denominator); a bf16 output adds half a step,
2^-8 of the value at most.  For a bf16 output over a bf16 cache, trees of more
than 64 rows (nodes times heads per KV head) hold their weights in one bf16:
half a step is 2^-8 of a weight, so the quotient of the two sums moves by at
most 2 2^-8 max |V|."""
import numpy as np
import pytest
import torch

import tree_reference as R

pytestmark = pytest.mark.gpu

BS = 16
E4M3 = R.e4m3_values()


@pytest.fixture(scope="module")
def pk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_21_gb300 as pk
    torch.cuda.set_device(0)
    return pk


@pytest.fixture(autouse=True)
def no_device_error(pk):
    yield
    assert pk.get_device_error()[0] == 0


class Case:
    """Inputs of one attention call.  lens include the nodes; unused slots and
    blocks of the pool hold NaN."""

    def __init__(self, lens, counts, Hq, Hkv, D, fp8=False, width=3, pads=0.0, seed=0,
                 chain=False, extra_rows=0, extra_blocks=3):
        rng = np.random.default_rng(seed)
        self.fp8, self.D, self.Hq, self.Hkv = fp8, D, Hq, Hkv
        self.lens, self.counts = np.asarray(lens), np.asarray(counts)
        B = len(lens)
        self.starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        T = int(self.starts[-1]) + extra_rows
        self.parents = np.concatenate([R.random_tree(rng, int(n), width, pads) for n in counts]
                                      + [np.full(extra_rows, -1, dtype=np.int32)]).astype(np.int32)
        self.chain = chain
        need = -(-self.lens // BS)
        self.NB = int(need.sum()) + extra_blocks
        perm = rng.permutation(self.NB)
        self.bt = np.full((B, max(1, int(need.max()) + 1)), -1, dtype=np.int32)
        at = 0
        for s in range(B):
            self.bt[s, :need[s]] = perm[at:at + need[s]]
            at += need[s]
        used = np.zeros((self.NB, BS), dtype=bool)
        for s in range(B):
            pos = np.arange(self.lens[s])
            used[self.bt[s, pos // BS], pos % BS] = True
        self.ks, self.vs = (0.011, 0.007) if fp8 else (1.0, 1.0)
        self.q = torch.from_numpy(rng.standard_normal((T, Hq, D))).to(torch.bfloat16)
        shape = (self.NB, Hkv, BS, D)
        unused = torch.from_numpy(~used)[:, None, :, None].expand(shape)
        if fp8:
            mk = lambda: torch.from_numpy(np.where(  # noqa: E731
                rng.random(shape) < 0.02, 0, rng.integers(0, 2, shape) * 128
                + rng.integers(0, 0x7f, shape)).astype(np.uint8))
            self.k, self.v = mk(), mk()
            # codes of magnitude up to 448: with ks the scores stay of order 1
            self.k = torch.where(self.k % 128 > 0x6f, self.k - 0x20, self.k)
            self.k[unused] = 0x7f
            self.v[unused] = 0xff
        else:
            self.k, self.v = (torch.from_numpy(rng.standard_normal(shape)).to(torch.bfloat16)
                              for _ in range(2))
            self.k[unused] = float("nan")
            self.v[unused] = float("nan")
        self.scale = D ** -0.5 / (4 if fp8 else 1)
        self.max_nodes = max(1, int(self.counts.max()) if B else 1)

    def values(self):
        if self.fp8:
            return E4M3[self.k.numpy()] * self.ks, E4M3[self.v.numpy()] * self.vs
        return self.k.double().numpy(), self.v.double().numpy()

    def reference(self):
        k, v = self.values()
        return R.attention(self.q.double().numpy(), k, v, self.bt, self.lens, self.starts,
                           None if self.chain else self.parents, self.scale)

    def device(self):
        c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return dict(q=self.q.cuda(), kc=self.k.cuda(), vc=self.v.cuda(), bt=c(self.bt),
                    lens=c(self.lens.astype(np.int32)), starts=c(self.starts),
                    parents=None if self.chain else c(self.parents))

    def run(self, pk, dtype=torch.bfloat16, t=None, out=None, ws=None, stream=None):
        t = t or self.device()
        if out is None:
            out = torch.full(self.q.shape, 7.0, dtype=dtype, device="cuda")
        if ws is None:
            ws = pk.alloc_tree_workspace(len(self.lens), self.max_nodes, self.Hq, self.Hkv, self.D,
                                         pk.FP8_E4M3 if self.fp8 else pk.BF16)
            ws.fill_(255)                         # NaN patterns: nothing may be read unwritten
        pk.paged_tree_attention(out, t["q"], t["kc"], t["vc"], t["bt"], t["lens"], t["starts"],
                                t["parents"], self.max_nodes, self.scale, ws, self.ks, self.vs,
                                stream=stream)
        return out

    def check(self, out, ref=None):
        ref = self.reference() if ref is None else ref
        n = int(self.starts[-1])
        got = out.double().cpu().numpy()
        _, v = self.values()
        vmax = np.nanmax(np.where(np.isfinite(v), np.abs(v), 0)) if v.size else 1.0
        tol = 2 * vmax * (2.0 ** -10 if self.fp8 else 2.0 ** -12)
        if out.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(ref)
            if not self.fp8:
                many = np.repeat(self.counts * (self.Hq // self.Hkv) > 64, self.counts)
                tol[:n] += (2 * 2.0 ** -8 * vmax * many)[:, None, None]
        assert np.isfinite(got[:n]).all()
        err = np.abs(got - ref)[:n]
        assert (err <= (tol if np.isscalar(tol) else tol[:n])).all(), float(err.max())
        assert (got[n:] == 7.0).all()             # rows behind the last sequence


HEADS = [(4, 1), (8, 8), (32, 8), (7, 1), (14, 2), (64, 1), (16, 1), (3, 3), (128, 1), (48, 2)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", HEADS)
def test_attention_matches_the_formula_for_every_head_layout(pk, heads, D, fp8):
    c = Case([37, 300, 5], [6, 11, 3], *heads, D, fp8, seed=heads[0] + D)
    ref = c.reference()
    for dtype in (torch.bfloat16, torch.float32):
        c.check(c.run(pk, dtype), ref)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 111, 112, 113, 127, 128, 129, 255, 1000])
def test_context_lengths_around_pages_and_tiles(pk, ctx, fp8):
    for counts in ([1, 1], [16, 2], [17, 9]):
        c = Case([ctx + n for n in counts], counts, 8, 2, 128, fp8, seed=ctx)
        c.check(c.run(pk, torch.float32))


@pytest.mark.parametrize("D,fp8", [(128, False), (64, False), (128, True), (64, True)])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 100, 127, 128])
def test_tree_sizes(pk, n, D, fp8):
    c = Case([n, n + 250], [n, n], 8, 2, D, fp8, seed=n)
    c.check(c.run(pk, torch.float32))


@pytest.mark.parametrize("heads", [(32, 8), (8, 8), (64, 4)])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_ragged_batch_with_empty_rows_sequences_and_padding(pk, heads, fp8):
    counts = np.array([5, 0, 1, 64, 9, 33, 2, 0, 12, 20])
    ctx = np.array([700, 0, 0, 130, 3, 2500, 16, 40, 95, 0])
    lens = ctx + counts
    lens[8] = 0                                   # nodes of a sequence without a context
    c = Case(lens, counts, *heads, 128, fp8, pads=0.3, seed=4, extra_rows=5)
    assert (c.parents == -2).any()
    c.check(c.run(pk))
    c.check(c.run(pk, torch.float32))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_the_most_rows_and_a_limit_above_the_trees(pk, D, fp8):
    c = Case([128, 300, 17], [128, 100, 1], 128, 1, D, fp8, seed=5)     # 16384 rows a KV head
    c.check(c.run(pk))
    c = Case([500, 40, 17], [3, 5, 1], 8, 2, D, fp8, seed=6)
    c.max_nodes = 128
    c.check(c.run(pk, torch.float32))


@pytest.mark.parametrize("fp8", [False, True])
def test_chains_need_no_parents(pk, fp8):
    c = Case([40, 500, 129], [8, 40, 1], 8, 2, 128, fp8, chain=True)
    c.check(c.run(pk, torch.float32))


@pytest.mark.parametrize("D", [64, 128])
def test_long_contexts_are_split_and_joined(pk, D):
    c = Case([9000, 20, 4100], [7, 3, 40], 8, 2, D, seed=2)
    c.check(c.run(pk, torch.float32))
    c = Case([20000], [4], 4, 1, D, True, seed=3)
    c.check(c.run(pk, torch.float32))


@pytest.mark.parametrize("D,fp8,heads", [(128, False, (8, 2)), (128, True, (8, 2)),
                                         (64, False, (16, 1)), (64, True, (64, 1))])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
def test_what_a_node_does_not_see_does_not_reach_it(pk, D, fp8, heads, bad):
    """A drafted token with non-finite K and V: it and its descendants see it,
    the other nodes' outputs are as if it held zeros."""
    if fp8 and bad != "nan":
        pytest.skip("E4M3 has no infinities")
    par = np.array([-1, 0, 0, 1, 2, 4, 0, -2, 6], dtype=np.int32)
    for ctx in (0, 9, 120, 400):
        c = Case([ctx + 9, ctx + 40], [9, 40], *heads, D, fp8, seed=ctx)
        c.parents[:9] = par
        clean = Case([ctx + 9, ctx + 40], [9, 40], *heads, D, fp8, seed=ctx)
        clean.parents[:9] = par
        for node in (2, 6):
            pos = ctx + node
            blk, off = c.bt[0, pos // BS], pos % BS
            for t, z in ((c.k, clean.k), (c.v, clean.v)):
                t[blk, :, off, 3::5] = 0x7f if fp8 else float(bad)
                z[blk, :, off] = 0
        out = c.run(pk, torch.float32).double().cpu().numpy()
        ref = clean.reference()
        seen = R.ancestors(par)
        good = [i for i in range(9) if not seen[i] & {2, 6}] + list(range(9, 49))
        tol = 2 * 10.0 * (2.0 ** -10 if fp8 else 2.0 ** -12)
        assert np.isfinite(out[good]).all()
        assert np.abs(out[good] - ref[good]).max() <= tol
        hit = [i for i in range(9) if seen[i] & {2, 6}]
        assert not np.isfinite(out[hit][:, :, 3::5]).any()


def test_a_non_finite_value_alone_reaches_its_own_columns(pk):
    """Finite keys, a drafted V row with inf and NaN elements: those who see it
    get inf and NaN in these columns, the right values in the others."""
    for D in (64, 128):
        c = Case([60], [10], 8, 2, D, seed=5, width=1)
        clean_v = c.v.clone()
        pos = 50 + 4
        blk, off = c.bt[0, pos // BS], pos % BS
        c.v[blk, 0, off, 1] = float("inf")
        c.v[blk, 0, off, 2] = float("-inf")
        c.v[blk, 1, off, 3] = float("nan")
        out = c.run(pk, torch.float32).double().cpu().numpy()
        c.v = clean_v
        ref = c.reference()
        assert np.isposinf(out[4:, :4, 1]).all() and np.isneginf(out[4:, :4, 2]).all()
        assert np.isnan(out[4:, 4:, 3]).all()
        ref[4:, :4, 1:3] = out[4:, :4, 1:3] = 0
        ref[4:, 4:, 3] = out[4:, 4:, 3] = 0
        assert np.abs(out - ref).max() <= 2 * 6 * 2.0 ** -12


def test_scales_of_either_sign_and_zero(pk):
    for scale in (-0.2, 0.0, 1.5):
        c = Case([70, 300], [9, 20], 8, 2, 128, seed=8)
        c.scale = scale
        # a larger scale scales the scores' error along: 1.5 sqrt(128) = 17 times
        out, ref = c.run(pk, torch.float32).double().cpu().numpy(), c.reference()
        assert np.abs(out - ref).max() <= 2 * 6 * 2.0 ** -12 * max(1, 17 * abs(scale) / 1.5)


def test_large_scores_move_the_running_maximum(pk):
    """Keys that grow along the context: every tile outgrows the one before."""
    c = Case([900, 260], [5, 30], 8, 2, 128, seed=9)
    for s, L in enumerate(c.lens):
        for pos in range(int(L)):
            c.k[c.bt[s, pos // BS], :, pos % BS] *= 1 + 0.05 * pos
    out, ref = c.run(pk, torch.float32).double().cpu().numpy(), c.reference()
    # scores up to 46 times larger: so is their error
    assert np.abs(out - ref).max() <= 46 * 2 * 6 * 2.0 ** -12


def test_one_root_is_a_decode_step(pk):
    for heads, D, fp8 in (((32, 8), 128, False), ((8, 8), 64, True), ((64, 1), 128, False)):
        c = Case([300, 17, 1, 2000], [1, 1, 1, 1], *heads, D, fp8, seed=11)
        t = c.device()
        got = c.run(pk, torch.float32, t)
        ref = torch.empty_like(got)
        dt = pk.FP8_E4M3 if fp8 else pk.BF16
        pk.paged_decode_attention(ref, t["q"], t["kc"], t["vc"], t["bt"], t["lens"], c.scale,
                                  pk.alloc_workspace(4, *heads, D, dt), c.ks, c.vs)
        c.check(got)
        c.check(ref)


def test_offsets_beyond_32_bits(pk):
    """Blocks at the far end of a cache of more than 2^31 elements."""
    NB, Hkv, D = 140000, 8, 128
    assert NB * Hkv * BS * D > 2 ** 31
    c = Case([90, 40], [9, 4], 16, Hkv, D, seed=12)
    t = c.device()
    far = torch.arange(NB - c.NB, NB, device="cuda")
    big = []
    for x in (t["kc"], t["vc"]):
        b = torch.empty((NB, Hkv, BS, D), dtype=x.dtype, device="cuda")
        b[far] = x
        big.append(b)
    t["kc"], t["vc"] = big
    t["bt"] = torch.where(t["bt"] >= 0, t["bt"] + (NB - c.NB), t["bt"])
    c.check(c.run(pk, torch.float32, t))


def test_repeated_calls_are_bit_identical_and_physical_places_do_not_matter(pk):
    a = Case([3000, 77, 500], [12, 3, 33], 16, 4, 128, seed=13)
    first = a.run(pk)
    assert all(torch.equal(first, a.run(pk)) for _ in range(3))
    b = Case([3000, 77, 500], [12, 3, 33], 16, 4, 128, seed=13, extra_blocks=9)
    perm = np.random.default_rng(1).permutation(b.NB)
    inv = torch.from_numpy(np.argsort(perm))
    k, v = torch.zeros_like(b.k), torch.zeros_like(b.v)
    k[:a.NB], v[:a.NB] = a.k, a.v
    b.k, b.v = k[inv], v[inv]
    b.bt = np.where(a.bt >= 0, perm[np.maximum(a.bt, 0)], -1).astype(np.int32)
    b.q, b.parents = a.q, a.parents
    assert torch.equal(first, b.run(pk))


@pytest.mark.parametrize("heads", [(8, 2), (32, 2)])
@pytest.mark.parametrize("B", [3, 90, 700])
def test_many_short_contexts_beside_long_ones(pk, heads, B):
    """Cuts of the work at every place: within a sequence, at its first page, and
    CTAs with many (sequence, KV head) pairs or none."""
    rng = np.random.default_rng(B)
    counts = rng.integers(0, 9, size=B)
    counts[B // 2] = 20
    ctx = np.where(rng.random(B) < 0.02, 3000, rng.integers(0, 40, size=B))
    ctx[0], ctx[-1] = 2100, 1500
    c = Case(ctx + counts, counts, *heads, 64, seed=B)
    ref = c.reference()
    for dtype in (torch.bfloat16, torch.float32):
        c.check(c.run(pk, dtype), ref)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_wait_that_runs_out_is_flagged_and_the_next_call_is_right(pk, fp8):
    """The hook's wait in the kernels for few and for many rows."""
    for counts in ([4, 3], [40, 33]):
        c = Case([900, 50], counts, 8, 2, 128, fp8, seed=21)
        pk.set_pipeline_stall(20000)               # ~10 us of SM clocks
        try:
            c.run(pk)
            torch.cuda.synchronize()
        finally:
            pk.set_pipeline_stall(0)
        assert pk.get_device_error()[0] == pk.DEVERR_PIPELINE_TIMEOUT
        c.check(c.run(pk, torch.float32))


@pytest.mark.parametrize("heads,n,fp8", [((32, 8), 8, False), ((32, 8), 30, False),
                                         ((32, 8), 64, False), ((16, 8), 20, True),
                                         ((32, 8), 48, True)])
def test_a_full_gpu_of_long_contexts(pk, heads, n, fp8):
    """Enough bytes that every copy takes its time: the 64-bit formula on the GPU
    for all rows, and the same bits from every call."""
    Hq, Hkv, D, B, L = heads[0], heads[1], 128, 24, 3000 + n
    gen = torch.Generator(device="cuda").manual_seed(n)
    nb = -(-L // BS)
    NB = B * nb
    bt = torch.randperm(NB, generator=gen, device="cuda").to(torch.int32).view(B, nb)
    x = [torch.randn((NB, Hkv, BS, D), generator=gen, device="cuda") for _ in range(2)]
    ks = vs = 1.0
    if fp8:
        ks, vs = 0.02, 0.03
        k, v = ((t / s).clamp(-448, 448).to(torch.float8_e4m3fn) for t, s in zip(x, (ks, vs)))
    else:
        k, v = (t.to(torch.bfloat16) for t in x)
    q = torch.randn((B * n, Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    rng = np.random.default_rng(n)
    par = np.concatenate([R.random_tree(rng, n, 3) for _ in range(B)]).astype(np.int32)
    starts = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    ws = pk.alloc_tree_workspace(B, n, Hq, Hkv, D, pk.FP8_E4M3 if fp8 else pk.BF16)
    dpar = torch.from_numpy(par).cuda()
    outs = []
    for _ in range(8):
        outs.append(torch.empty((B * n, Hq, D), dtype=torch.float32, device="cuda"))
        pk.paged_tree_attention(outs[-1], q, k, v, bt, lens, starts, dpar, n, D ** -0.5, ws, ks, vs)
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    G = Hq // Hkv
    for s in range(B):
        K, V = (t[bt[s].long()].double().transpose(0, 1).reshape(Hkv, -1, D)[:, :L] * z
                for t, z in ((k, ks), (v, vs)))
        Q = q[s * n:(s + 1) * n].double().view(n, Hkv, G, D).transpose(0, 1).reshape(Hkv, n * G, D)
        mask = torch.zeros((n, L), dtype=torch.float64)
        mask[:, L - n:] = -np.inf
        for i, seen in enumerate(R.ancestors(par[s * n:(s + 1) * n])):
            mask[i, [L - n + j for j in seen]] = 0
        w = torch.softmax(Q @ K.transpose(1, 2) * D ** -0.5
                          + mask.cuda().repeat_interleave(G, 0)[None], -1)
        ref = (w @ V).view(Hkv, n, G, D).transpose(0, 1).reshape(n, Hq, D)
        tol = 2 * float(V.abs().max()) * (2.0 ** -10 if fp8 else 2.0 ** -12)
        assert float((outs[0][s * n:(s + 1) * n].double() - ref).abs().max()) <= tol


def test_two_streams_and_two_captured_graphs(pk):
    cases = [Case([2500, 400], [20, 5], 16, 4, 128, seed=14),
             Case([90, 4000], [3, 64], 32, 8, 128, True, seed=15)]
    state = [(c, c.device(), c.run(pk), pk.alloc_tree_workspace(
        2, c.max_nodes, c.Hq, c.Hkv, c.D, pk.FP8_E4M3 if c.fp8 else pk.BF16)) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(s[2]) for s in state]
    for _ in range(20):
        for st, (c, t, _, ws), o in zip(streams, state, outs):
            c.run(pk, t=t, out=o, ws=ws, stream=st)
    torch.cuda.synchronize()
    for (_, _, want, _), o in zip(state, outs):
        assert torch.equal(want, o)
    graphs = []
    for (c, t, _, ws), o in zip(state, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(pk, t=t, out=o, ws=ws)
        graphs.append(g)
    # other inputs in the captured buffers: shorter contexts, another tree, other queries
    for c, t, _, _ in state:
        c.lens = c.lens - 37
        c.parents = np.concatenate([R.random_tree(np.random.default_rng(3), int(n), 2)
                                    for n in c.counts]).astype(np.int32)
        c.q = c.q.flip(0)
        t["lens"].copy_(torch.from_numpy(c.lens.astype(np.int32)))
        t["parents"].copy_(torch.from_numpy(c.parents))
        t["q"].copy_(c.q)
    for o in outs:
        o.fill_(7.0)
    for st, g in zip(streams, graphs):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    for (c, _, _, _), o in zip(state, outs):
        c.check(o)


def test_tables_in_pinned_host_memory(pk):
    c = Case([300, 40], [9, 4], 8, 2, 128, seed=16)
    t = c.device()
    want = c.run(pk, t=t)
    for key in ("bt", "lens", "starts", "parents", "q"):
        t[key] = t[key].cpu().pin_memory()
    out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16).pin_memory()
    c.run(pk, t=t, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want.cpu())


def test_bad_tables_are_flagged_and_leave_the_other_sequences_alone(pk):
    def run(change):
        c = Case([300, 90, 200], [9, 4, 20], 8, 2, 128, seed=17)
        t = c.device()
        change(c, t)
        out = c.run(pk, torch.float32, t)
        torch.cuda.synchronize()
        flags, detail = pk.get_device_error()
        got, ref = out.double().cpu().numpy(), c.reference()
        ok = [np.abs(got[a:b] - ref[a:b]).max() < 2 * 6 * 2.0 ** -12
              for a, b in ((0, 9), (9, 13), (13, 33))]
        return flags, detail, ok

    def block(c, t):
        t["bt"][1, 2] = c.NB

    def neg(c, t):
        t["bt"][1, 0] = -1

    def long(c, t):
        t["lens"][2] = 16 * c.bt.shape[1] + 1

    def parent(c, t):
        t["parents"][9 + 2] = 3

    def parent_low(c, t):
        t["parents"][9 + 2] = -7

    def short(c, t):
        t["lens"][1] = 2

    assert run(lambda c, t: None) == (0, -1, [True] * 3)
    f, d, ok = run(block)
    assert f == pk.DEVERR_BLOCK_OUT_OF_RANGE and ok[0] and ok[2]
    f, d, ok = run(neg)
    assert f == pk.DEVERR_BLOCK_OUT_OF_RANGE and d == -1 and ok[0] and ok[2]
    f, d, ok = run(long)
    assert f & pk.DEVERR_CONTEXT_TOO_LONG and ok[0] and ok[1]
    f, d, ok = run(parent)
    assert (f, d) == (pk.DEVERR_BAD_TREE, 3) and ok[0] and ok[2]
    f, d, ok = run(parent_low)
    assert (f, d) == (pk.DEVERR_BAD_TREE, -7) and ok[0] and ok[2]
    f, d, ok = run(short)
    assert (f, d) == (pk.DEVERR_BAD_TREE, 2) and ok[0] and ok[2]
    # starts: sequence 1 would have more nodes than max_nodes, and 2 a negative number
    c = Case([300, 90, 200], [9, 4, 20], 8, 2, 128, seed=17)
    t = c.device()
    ref = c.reference()
    t["starts"].copy_(torch.tensor([0, 9, 33, 13], dtype=torch.int32))
    out = c.run(pk, torch.float32, t)
    torch.cuda.synchronize()
    assert pk.get_device_error()[0] == pk.DEVERR_BAD_TREE
    got = out.double().cpu().numpy()
    assert np.abs(got[:9] - ref[:9]).max() < 2 * 6 * 2.0 ** -12 and (got[9:] == 7.0).all()


def test_a_workspace_that_is_too_small_is_refused(pk):
    c = Case([300], [9], 8, 2, 128)
    t = c.device()
    ws = pk.alloc_tree_workspace(1, 9, 8, 2, 128)
    with pytest.raises(pk.KVError) as e:
        c.run(pk, t=t, ws=ws[:ws.numel() - 1])
    assert e.value.code == pk.KV_ERR_INVALID_ARG


# ------------------------------------------------------------------ verification

class Verify:
    def __init__(self, counts, V, width=2, seed=0, bf16=False, noise=0.5, pads=0.0, sharp=1.5):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.counts = np.asarray(counts)
        B = len(counts)
        self.starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        T = int(self.starts[-1])
        self.parents = (np.concatenate([R.random_tree(rng, int(n), width, pads) for n in counts])
                        if T else np.zeros(0)).astype(np.int32)
        dt = torch.bfloat16 if bf16 else torch.float32
        logits = torch.randn((T, V), generator=g) * sharp
        self.target = torch.softmax(logits, 1).to(dt)
        self.draft = torch.softmax(logits + noise * torch.randn((T, V), generator=g), 1).to(dt)
        at = np.maximum(self.parents, 0) + np.repeat(self.starts[:-1], self.counts)
        self.tokens = (torch.multinomial(self.draft[at].float() + 1e-30, 1, generator=g)[:, 0]
                       .numpy().astype(np.int32) if T else np.zeros(0, np.int32))
        self.u, self.su = torch.rand(T, generator=g).numpy(), torch.rand(B, generator=g).numpy()
        self.max_nodes = max(1, int(self.counts.max()))

    def run(self, pk, draft=True, greedy=False, chain=False, target=None, dprob=None):
        c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        B = len(self.counts)
        al = torch.full((B,), 99, dtype=torch.int32, device="cuda")
        an = torch.full((B, self.max_nodes), 99, dtype=torch.int32, device="cuda")
        ot = torch.full((B, self.max_nodes), 99, dtype=torch.int32, device="cuda")
        target = self.target.cuda() if target is None else target
        dprob = self.draft.cuda() if dprob is None else dprob
        pk.kv_tree_verify(al, an, ot, target, c(self.tokens),
                          None if chain else c(self.parents), c(self.starts),
                          None if greedy else c(self.u), None if greedy else c(self.su),
                          draft_probs=dprob if draft else None, greedy=greedy)
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in (al, an, ot)]

    def check(self, pk, draft=True, greedy=False, chain=False, **kw):
        got = self.run(pk, draft, greedy, chain, **kw)
        want = R.verify(self.target.double().numpy(), self.draft.double().numpy() if draft else None,
                        self.tokens, None if chain else self.parents, self.starts, self.u, self.su,
                        self.max_nodes, greedy)
        for g, w in zip(got, want):
            assert np.array_equal(g, w)
        return got


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 31, 127, 128, 1000, 4097, 50001])
def test_verify_over_vocabularies(pk, V, bf16):
    for draft in (True, False):
        v = Verify([6, 1, 0, 17, 9], V, 3, seed=V, bf16=bf16)
        v.check(pk, draft)
    v.check(pk, greedy=True)


@pytest.mark.parametrize("width", [1, 2, 5])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_many_trees(pk, width, draft):
    """Refusals of one, several and all children, at 200 trees each."""
    rng = np.random.default_rng(width)
    for noise in (0.1, 1.0, 3.0):
        v = Verify(rng.integers(1, 40, size=200), 300, width, seed=width, noise=noise, pads=0.05)
        lens, _, _ = v.check(pk, draft)
        # chosen tokens are as unlikely as any of the 300: they are hardly ever accepted
        assert lens.min() >= 1 and (not draft or lens.max() >= 2)


def test_verify_chains_and_the_largest_tree(pk):
    v = Verify([128, 5, 128], 600, 1, seed=3, noise=0.02, sharp=0.3)
    got = v.check(pk, chain=True)
    assert got[0].max() > 10
    for a, b in zip(got, v.run(pk)):
        assert np.array_equal(a, b)
    v = Verify([128, 128], 600, 40, seed=4)
    v.check(pk)
    v.check(pk, draft=False)


def test_verify_strides_and_alignments(pk):
    v = Verify([9, 4, 12], 1003, 3, seed=5)
    for bf16 in (False, True):
        if bf16:
            v.target, v.draft = v.target.to(torch.bfloat16), v.draft.to(torch.bfloat16)
        want = v.run(pk)
        for ts, ds, to, do in ((1003, 1003, 0, 0), (1008, 1008, 0, 0), (1008, 1008, 1, 1),
                               (1011, 1008, 0, 0), (1016, 1024, 3, 2), (2048, 1005, 5, 0)):
            bufs = []
            for p, st, off in ((v.target, ts, to), (v.draft, ds, do)):
                b = torch.full((25 * st + 16,), float("nan"), dtype=p.dtype, device="cuda")
                view = b[off:off + 25 * st].view(25, st)[:, :1003]
                view.copy_(p)
                bufs.append(view)
            for g, w in zip(v.run(pk, target=bufs[0], dprob=bufs[1]), want):
                assert np.array_equal(g, w)
            for g, w in zip(v.run(pk, target=bufs[0], draft=False), v.run(pk, draft=False)):
                assert np.array_equal(g, w)
        v.check(pk)


def test_verify_edge_values(pk):
    # numbers at the ends of [0, 1)
    v = Verify([7] * 60, 200, 3, seed=6)
    v.u[::3], v.u[1::3] = 0.0, np.float32(1 - 2.0 ** -24)
    v.su[::2], v.su[1::2] = 0.0, np.float32(1 - 2.0 ** -24)
    v.check(pk)
    v.check(pk, draft=False)
    # what does not count: NaN, infinite and negative entries; all of a row
    v = Verify([7] * 60, 200, 3, seed=7)
    rng = np.random.default_rng(7)
    for p in (v.target, v.draft):
        hit = torch.from_numpy(rng.random(p.shape) < 0.2)
        what = torch.tensor([float("nan"), float("inf"), -1.0, float("-inf"), -0.0, 1e-42])
        p[hit] = what[torch.from_numpy(rng.integers(0, 6, int(hit.sum())))]
    v.target[3::7] = 0.0
    v.check(pk)
    v.check(pk, draft=False)
    # target equal to draft: nothing is left once a token of probability zero is refused
    v = Verify([5] * 30, 50, 2, seed=8)
    v.target[:, 25:] = 0.0
    v.draft = v.target.clone()
    v.tokens[1::2] = 40
    v.check(pk)
    # tokens outside the vocabulary are never accepted; the same token twice
    v = Verify([9] * 30, 50, 4, seed=9)
    v.tokens[2::9], v.tokens[5::9] = -3, 50
    v.tokens[3::9] = v.tokens[4::9]
    v.check(pk)
    v.check(pk, draft=False)
    v.check(pk, greedy=True)


def test_verify_greedy_on_logits(pk):
    v = Verify([12] * 40, 777, 3, seed=10)
    v.target = torch.randn((480, 777), generator=torch.Generator().manual_seed(1))
    v.target[5::11, 100:] = float("nan")
    v.target[7::13, 3] = v.target[7::13, 500] = 9.0          # ties: the lowest index
    v.target[9::17] = float("-inf")
    top = torch.where(v.target.isnan(), torch.tensor(float("-inf")), v.target).argmax(1).numpy()
    at = np.maximum(v.parents, 0) + np.repeat(v.starts[:-1], v.counts)
    take = np.random.default_rng(2).random(480) < 0.6
    v.tokens = np.where(take, top[at], v.tokens).astype(np.int32)
    lens, _, _ = v.check(pk, greedy=True)
    assert lens.max() > 2
    v.target = v.target.to(torch.bfloat16)
    v.check(pk, greedy=True)


def test_verify_bad_tables_are_flagged(pk):
    v = Verify([5, 6, 7], 64, 2, seed=11)
    want = v.run(pk)
    v.parents[5 + 3] = 4                          # sequence 1: a parent behind its node
    got = v.run(pk)
    assert pk.get_device_error() == (pk.DEVERR_BAD_TREE, 4)
    for g, w in zip(got, want):
        assert np.array_equal(g[[0, 2]], w[[0, 2]])
    v.parents[5 + 3] = -1
    v.starts[2] = 4                               # sequence 1: a negative number of nodes
    got = v.run(pk)
    assert pk.get_device_error()[0] == pk.DEVERR_BAD_TREE
    assert got[0][1] == 0 and (got[1][1] == -1).all() and (got[2][1] == -1).all()
    assert np.array_equal(got[1][0], want[1][0])


def test_verify_captured_and_replayed_with_other_numbers(pk):
    v = Verify([9] * 20, 5000, 3, seed=12)
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    out = [torch.zeros(20, dtype=torch.int32, device="cuda")] + [
        torch.zeros((20, 9), dtype=torch.int32, device="cuda") for _ in range(2)]
    tg, dr, tok, par, st, u, su = (v.target.cuda(), v.draft.cuda(), c(v.tokens), c(v.parents),
                                   c(v.starts), c(v.u), c(v.su))
    pk.kv_tree_verify(*out, tg, tok, par, st, u, su, draft_probs=dr)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.kv_tree_verify(*out, tg, tok, par, st, u, su, draft_probs=dr)
    w = Verify([9] * 20, 5000, 3, seed=13)
    for dst, src in ((tg, w.target), (dr, w.draft), (tok, torch.from_numpy(w.tokens)),
                     (par, torch.from_numpy(w.parents)), (u, torch.from_numpy(w.u)),
                     (su, torch.from_numpy(w.su))):
        dst.copy_(src)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, w.check(pk)):
        assert np.array_equal(a.cpu().numpy(), b)


# -------------------------------------------------------------------- compaction

def _compact_case(rng, B, n_hi, layers, Hkv, D, dtype):
    counts = rng.integers(0, n_hi + 1, size=B)
    lens = rng.integers(0, 70, size=B) + counts
    need = -(-lens // BS)
    NB = int(need.sum()) + 2
    perm = rng.permutation(NB)
    bt = np.full((B, int(need.max()) + 1), -1, dtype=np.int32)
    at = 0
    for s in range(B):
        bt[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    nodes = np.full((B, n_hi), -1, dtype=np.int32)
    accept = np.array([rng.integers(0, n + 1) for n in counts], dtype=np.int32)
    for s in range(B):
        nodes[s, :accept[s]] = np.sort(rng.permutation(counts[s])[:accept[s]])
    lo = 0 if dtype == np.uint8 else -32768
    caches = rng.integers(lo, 255 if dtype == np.uint8 else 32767,
                          size=(2, layers, NB, Hkv, BS, D)).astype(dtype)
    return counts, lens, bt, starts, nodes, accept, caches


@pytest.mark.parametrize("dtype", [np.int16, np.uint8])
@pytest.mark.parametrize("B,n_hi,layers,Hkv,D", [(1, 8, 1, 1, 64), (5, 128, 2, 3, 64),
                                                 (9, 30, 5, 8, 128), (3, 20, 130, 1, 128),
                                                 (40, 12, 3, 2, 64), (2, 60, 2, 2, 48)])
def test_compaction_moves_the_accepted_nodes_and_nothing_else(pk, B, n_hi, layers, Hkv, D, dtype):
    rng = np.random.default_rng(B + D)
    counts, lens, bt, starts, nodes, accept, caches = _compact_case(rng, B, n_hi, layers, Hkv, D,
                                                                    dtype)
    dev = torch.from_numpy(caches).cuda()
    typed = dev.view(torch.bfloat16) if dtype == np.int16 else dev
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()  # noqa: E731
    pk.kv_tree_compact(pk.CacheLayers(list(typed[0]), list(typed[1])), c(bt), c(lens), c(starts),
                       c(nodes), c(accept))
    got = dev.cpu().numpy()
    for l in range(layers):
        k, v = R.compact(caches[0, l], caches[1, l], bt, lens, starts, nodes, accept)
        assert np.array_equal(got[0, l], k) and np.array_equal(got[1, l], v)


def test_compaction_of_more_sequences_than_run_at_once_and_replayed(pk):
    rng = np.random.default_rng(8)
    counts, lens, bt, starts, nodes, accept, caches = _compact_case(rng, 1300, 6, 1, 2, 64, np.int16)
    dev = torch.from_numpy(caches).cuda()
    typed = dev.view(torch.bfloat16)
    layers = pk.CacheLayers(list(typed[0]), list(typed[1]))
    t = [torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()
         for a in (bt, lens, starts, nodes, accept)]
    zero = torch.zeros_like(t[4])
    pk.kv_tree_compact(layers, *t[:4], zero)       # nothing accepted, nothing moves
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.kv_tree_compact(layers, *t)
    assert np.array_equal(dev.cpu().numpy(), caches)
    g.replay()
    torch.cuda.synchronize()
    got = dev.cpu().numpy()
    k, v = R.compact(caches[0, 0], caches[1, 0], bt, lens, starts, nodes, accept)
    assert np.array_equal(got[0, 0], k) and np.array_equal(got[1, 0], v)


def test_compaction_leaves_out_paths_and_blocks_that_break_the_rules(pk):
    rng = np.random.default_rng(5)
    for what in ("order", "range", "length", "block", "context"):
        counts, lens, bt, starts, nodes, accept, caches = _compact_case(rng, 3, 10, 2, 2, 64,
                                                                        np.int16)
        counts[:] = 10
        starts = np.arange(4, dtype=np.int32) * 10
        lens = np.array([30, 45, 20])
        bt = np.arange(12, dtype=np.int32).reshape(3, 4)
        nodes[:] = -1
        nodes[:, :4] = [0, 3, 5, 9]
        accept[:] = 4
        caches = rng.integers(-32768, 32767, size=(2, 2, 12, 2, BS, 64)).astype(np.int16)
        ok_nodes, ok_accept = nodes.copy(), accept.copy()
        flag = pk.DEVERR_BAD_TREE
        if what == "order":
            nodes[1, :4] = [0, 5, 3, 9]
        elif what == "range":
            nodes[1, 3] = 10
        elif what == "length":
            accept[1] = 11
        elif what == "context":
            lens[1] = 9
        else:
            bt[1, 2] = 12                          # positions 32..47 of sequence 1
            flag = pk.DEVERR_BLOCK_OUT_OF_RANGE
        ok_accept[1] = 0
        dev = torch.from_numpy(caches).cuda()
        typed = dev.view(torch.bfloat16)
        c = lambda a: torch.from_numpy(  # noqa: E731
            np.ascontiguousarray(a).astype(np.int32)).cuda()
        pk.kv_tree_compact(pk.CacheLayers(list(typed[0]), list(typed[1])), c(bt), c(lens),
                           c(starts), c(nodes), c(accept))
        torch.cuda.synchronize()
        assert pk.get_device_error()[0] == flag
        got = dev.cpu().numpy()
        if what == "block":
            lens[1], bt[1, 2] = 45, 6
        for l in range(2):
            k, v = R.compact(caches[0, l], caches[1, l], bt, lens, starts, ok_nodes, ok_accept)
            assert np.array_equal(got[0, l], k) and np.array_equal(got[1, l], v), what


# ------------------------------------------------------------------ all of them

@pytest.mark.parametrize("fp8", [False, True])
def test_a_run_of_steps_as_a_program_uses_them(pk, fp8):
    """Three steps of a two-layer batch: reserve, append, attend, verify, compact,
    truncate.  After each the caches hold exactly the accepted tokens' K and V,
    and what the next step's attention returns is the formula over them."""
    rng = np.random.default_rng(21)
    B, Hq, Hkv, D, layers, V, NB = 4, 8, 2, 64, 2, 97, 80
    ks, vs = (0.02, 0.02) if fp8 else (1.0, 1.0)
    alloc = pk.BlockAllocator(NB, Hkv, D, pk.FP8_E4M3 if fp8 else pk.BF16)
    dt = torch.uint8 if fp8 else torch.bfloat16
    kc = [torch.zeros((NB, Hkv, BS, D), dtype=dt, device="cuda") for _ in range(layers)]
    vc = [torch.zeros_like(kc[0]) for _ in range(layers)]
    caches = pk.CacheLayers(kc, vc)
    ids = list(range(B))
    for i in (0, 1, 2):
        alloc.add(i, 0)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).cuda()  # noqa: E731
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    held = [[[] for _ in range(B)] for _ in range(layers)]       # accepted (k, v) per sequence
    # prompts by chains, then sequence 3 branches off sequence 0
    slots, bt, lens, starts, _ = alloc.tree_step([0, 1, 2], [21, 5, 40], 8)
    for l in range(layers):
        k, v = bf(66, Hkv, D), bf(66, Hkv, D)
        pk.kv_append(k, v, kc[l], vc[l], c(slots), ks, vs)
        for s in range(3):
            held[l][s] = [(k[i], v[i]) for i in range(starts[s], starts[s + 1])]
        held[l][3] = held[l][0][:19]
    alloc.fork(0, 3, 19)
    copied = 0
    for step in range(3):
        counts = rng.integers(1, 20, size=B)
        slots, bt, lens, starts, (src, dst) = alloc.tree_step(ids, counts, 12)
        copied += len(src)
        if len(src):
            for l in range(layers):
                pk.kv_copy_blocks(kc[l], vc[l], c(src), c(dst))
        T = int(starts[-1])
        parents = np.concatenate([R.random_tree(rng, int(n), 2) for n in counts]).astype(np.int32)
        ws = pk.alloc_tree_workspace(B, 20, Hq, Hkv, D, pk.FP8_E4M3 if fp8 else pk.BF16)
        dbt, dl, ds, dp = c(bt), c(lens), c(starts), c(parents)
        new = []
        for l in range(layers):
            q, k, v = bf(T, Hq, D), bf(T, Hkv, D), bf(T, Hkv, D)
            new.append((k, v))
            pk.kv_append(k, v, kc[l], vc[l], c(slots), ks, vs)
            out = torch.empty((T, Hq, D), dtype=torch.float32, device="cuda")
            pk.paged_tree_attention(out, q, kc[l], vc[l], dbt, dl, ds, dp, 20, D ** -0.5, ws, ks,
                                    vs)
            # the formula over the accepted tokens and the new ones, laid out afresh
            quant = (lambda x, s: torch.from_numpy(E4M3[np.minimum(  # noqa: E731
                (x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                .cpu().numpy(), 255)]) * s) if fp8 else (lambda x, s: x.double().cpu())
            for s in range(B):
                a, b = int(starts[s]), int(starts[s + 1])
                seq = held[l][s] + [(k[i], v[i]) for i in range(a, b)]
                nb = -(-len(seq) // BS)
                K, W = (torch.zeros((nb * BS, Hkv, D), dtype=torch.float64) for _ in range(2))
                K[:len(seq)] = quant(torch.stack([x[0] for x in seq]), ks)
                W[:len(seq)] = quant(torch.stack([x[1] for x in seq]), vs)
                K, W = (x.reshape(nb, BS, Hkv, D).transpose(1, 2).numpy() for x in (K, W))
                ref = R.attention(q[a:b].double().cpu().numpy(), K, W,
                                  np.arange(nb, dtype=np.int32)[None], [len(seq)], [0, b - a],
                                  parents[a:b], D ** -0.5)
                tol = 2 * np.abs(W).max() * (2.0 ** -10 if fp8 else 2.0 ** -12)
                assert np.abs(out[a:b].double().cpu().numpy() - ref).max() <= tol
        ver = Verify(counts, V, 2, seed=step, noise=0.2)
        ver.parents, ver.max_nodes = parents, 20
        al, an, ot = ver.check(pk)
        pk.kv_tree_compact(caches, dbt, dl, ds, c(an), c(al))
        base = lens - counts
        alloc.truncate(ids, base + al)
        for l in range(layers):
            for s in range(B):
                held[l][s] = held[l][s] + [(new[l][0][starts[s] + i], new[l][1][starts[s] + i])
                                           for i in an[s, :al[s]]]
        assert [r["len"] for r in alloc.trace(ids)] == [len(h) for h in held[0]]
    assert copied >= 1
