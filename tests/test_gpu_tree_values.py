"""Draft-tree attention and its neighbours on the GPU, where a result can be lost without a
fault: infinities and NaN that a node sees, queries of every magnitude, workspaces of another
size, idle rows, single lost keys in bf16 outputs, numbers at the border of two tokens.

Where nothing else is said, the tolerances are those of test_gpu_tree.py."""
import numpy as np
import pytest
import torch

import tree_reference as R
from test_gpu_tree import BS, Case

pytestmark = pytest.mark.gpu


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


def reference(c):
    with np.errstate(all="ignore"):
        return c.reference()


def same(c, out, ref):
    """Every column: NaN where the formula has NaN, the same infinities, and the formula's
    value elsewhere."""
    n = int(c.starts[-1])
    got, ref = out.double().cpu().numpy()[:n], ref[:n]
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isposinf(got), np.isposinf(ref))
    assert np.array_equal(np.isneginf(got), np.isneginf(ref))
    _, v = c.values()
    vmax = np.nanmax(np.where(np.isfinite(v), np.abs(v), 0))
    tol = 2 * vmax * (2.0 ** -10 if c.fp8 else 2.0 ** -12)
    ok = np.isfinite(ref)
    assert np.abs(got[ok] - ref[ok]).max(initial=0) <= tol


# nodes of the trees, heads: up to 32 and 64 rows, one tile, two tiles, two teams of CTAs
ROWS = [([9, 5], (8, 2)), ([16, 3], (8, 2)), ([20, 1], (8, 2)), ([40, 7], (8, 2)),
        ([72, 9], (16, 2))]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts,heads", ROWS)
@pytest.mark.parametrize("ctx", [0, 9, 400, 5000])
def test_a_nan_query_gives_nan(pk, ctx, counts, heads, D, fp8):
    """In every column of its own row, and in no other row; a padding node stays zero."""
    c = Case([ctx + counts[0], 30 + counts[1]], counts, *heads, D, fp8, seed=ctx + counts[0])
    c.parents[counts[0] - 1] = -2
    c.q[2, 1, D // 2] = float("nan")
    c.q[2, heads[0] - 1] = float("nan")
    c.q[counts[0] - 2, 0, 3] = float("nan")
    c.q[counts[0] - 1, 2, 0] = float("nan")
    ref = reference(c)
    assert np.isnan(ref[2, 1]).all() and (ref[counts[0] - 1] == 0).all()
    same(c, c.run(pk, torch.float32), ref)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts,heads", ROWS)
@pytest.mark.parametrize("ctx", [0, 9, 400, 5000])
def test_a_nan_key_gives_nan_to_the_nodes_that_see_it(pk, ctx, counts, heads, D, fp8):
    """Finite values.  A drafted token with a NaN key: its descendants; a committed one: every
    node of its sequence, in the heads of its KV head."""
    for what in ("drafted", "committed"):
        if what == "committed" and ctx == 0:
            continue
        c = Case([ctx + counts[0], 30 + counts[1]], counts, *heads, D, fp8, seed=ctx + counts[0])
        pos = ctx + 2 if what == "drafted" else ctx // 2
        c.k[c.bt[0, pos // BS], 0, pos % BS, 5] = 0x7f if fp8 else float("nan")
        ref = reference(c)
        half = heads[0] // heads[1]
        assert np.isnan(ref[2, :half]).all() and np.isfinite(ref[:, half:]).all()
        same(c, c.run(pk, torch.float32), ref)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts,heads", ROWS)
@pytest.mark.parametrize("ctx", [0, 9, 400, 5000])
def test_infinite_queries_follow_the_formula(pk, ctx, counts, heads, D, fp8):
    """Scores of infinities of one sign or both; where a node sees only scores of -inf, the
    softmax is NaN."""
    c = Case([ctx + counts[0], 30 + counts[1]], counts, *heads, D, fp8, seed=ctx + counts[0])
    c.parents[counts[0] - 1] = -2
    # element 3 of every key of KV head 0 is negative, element 4 of both signs
    if fp8:
        c.k[:, 0, :, 3] |= 0x80
        c.k[:, 0, :, 3][c.k[:, 0, :, 3] == 0x80] = 0x90
    else:
        c.k[:, 0, :, 3] = -c.k[:, 0, :, 3].abs()
    c.q[1, 0, 3] = float("inf")
    c.q[2, 1, 3] = float("-inf")
    c.q[3, 0, 4] = float("inf")
    c.q[counts[0] - 1, 0, 4] = float("inf")
    ref = reference(c)
    assert np.isnan(ref[1:3].diagonal()).all() and (ref[counts[0] - 1] == 0).all()
    same(c, c.run(pk, torch.float32), ref)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts,heads", ROWS)
@pytest.mark.parametrize("ctx", [0, 9, 400, 5000])
def test_infinite_keys_follow_the_formula(pk, ctx, counts, heads, D):
    c = Case([ctx + counts[0], 30 + counts[1]], counts, *heads, D, seed=ctx + counts[0])
    for pos in {ctx // 3, ctx + 1}:
        c.k[c.bt[0, pos // BS], 0, pos % BS, 7] = float("inf")
    ref = reference(c)
    same(c, c.run(pk, torch.float32), ref)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_limits_workspace_serves_every_smaller_call(pk, fp8):
    dt = pk.FP8_E4M3 if fp8 else pk.BF16
    for D in (64, 128):
        for G in (1, 2, 3, 4, 5, 7, 8, 16, 24, 33, 64, 65, 128):
            sizes = [pk.tree_workspace_bytes(4, n, G, 1, D, dt) for n in range(1, 129)]
            assert sizes == sorted(sizes), (D, G)
    ws = pk.alloc_tree_workspace(2, 96, 16, 2, 128, dt)
    for counts in ([64, 5], [40, 33], [8, 4]):
        c = Case([300 + counts[0], 2000 + counts[1]], counts, 16, 2, 128, fp8, seed=counts[0])
        ws.fill_(255)
        c.check(c.run(pk, torch.float32, ws=ws))


def scored(c):
    """The formula's outputs, sum_j w_j |V_j| beside them, and of each row the scores of
    all keys it sees, their values, and the largest |q_d k_d| times the scale."""
    k, v = c.values()
    q = c.q.double().numpy()
    out, mean = np.zeros_like(q), np.zeros_like(q)
    scores, top = {}, np.zeros(q.shape[:2])
    G = c.Hq // c.Hkv
    for s in range(len(c.lens)):
        t0, n, L = int(c.starts[s]), int(c.counts[s]), int(c.lens[s])
        pages = c.bt[s, :-(-L // BS)]
        K, V = (x[pages].transpose(1, 0, 2, 3).reshape(c.Hkv, -1, c.D)[:, :L] for x in (k, v))
        for i, seen in enumerate(R.ancestors(c.parents[t0:t0 + n])):
            idx = np.concatenate([np.arange(L - n), L - n + np.array(sorted(seen), dtype=int)])
            for h in range(c.Hq):
                x = K[h // G, idx] @ q[t0 + i, h] * c.scale
                w = np.exp(x - x.max())
                out[t0 + i, h] = w @ V[h // G, idx] / w.sum()
                mean[t0 + i, h] = w @ np.abs(V[h // G, idx]) / w.sum()
                scores[t0 + i, h] = x, V[h // G, idx]
                top[t0 + i, h] = np.abs(K[h // G, idx] * q[t0 + i, h]).max() * abs(c.scale)
    return out, mean, scores, top


def check_magnitudes(c, got, weight, score, element):
    """Outputs of scores that are off by d at most, d = score * the largest product + element
    * the sum of a row's element errors, and of weights that are off by `weight` of theirs:
    by at most (weight + 2 (e^d - 1)) sum_j w_j |V_j|; where d is large, but the largest score
    so far above the others that its weight is 1, that key's value."""
    ref, mean, scores, top = scored(c)
    assert np.isfinite(got).all()
    q = c.q.double().numpy()
    close = sharp = 0
    for (t, h), (x, V) in scores.items():
        d = score * top[t, h] + element * np.abs(q[t, h]).max()
        two = np.sort(x)[-2:] if len(x) > 1 else np.array([-np.inf, x[0]])
        if d < 0.05:
            bound = (weight + 2 * np.expm1(d)) * mean[t, h] + 2.0 ** -22
            close += 1
        elif two[1] - two[0] > 2 * d + 30:       # the other weights together: len(x) e^-30
            bound = weight * mean[t, h] + len(x) * np.exp(-30) * np.abs(V).max()
            sharp += 1
        else:
            continue
        assert (np.abs(got[t, h] - ref[t, h]) <= bound).all(), (t, h, d)
    assert close + sharp > 0.95 * len(scores) and sharp > 0


def magnitudes(counts, heads, D, fp8):
    """Query rows of normal values times a power of two of their own, from the subnormals to
    the largest, one row whose elements each have their own, and one with the largest."""
    c = Case([300, 900 + counts[1]], counts, *heads, D, fp8, seed=3)
    if fp8:
        c.ks *= 2.0 ** -20
    else:
        c.k = (c.k.float() * 2.0 ** -20).to(torch.bfloat16)
    rng = np.random.default_rng(7)
    q = c.q.double().numpy()
    q *= np.exp2(rng.choice([0, 17, 20, 23, 26, 40, 100, 124, -20, -130], size=q.shape[:2]))[..., None]
    q[0, 1] = np.exp2(rng.integers(-130, 124, size=D)) * np.sign(q[0, 1])
    q[1, 1, 5] = 3e38
    c.q = torch.from_numpy(q).to(torch.bfloat16)
    assert torch.isfinite(c.q.float()).all()
    return c


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts,heads", ROWS)
def test_query_magnitudes_over_the_whole_bf16_range(pk, counts, heads, D):
    """Scores up to 10^32.  A float32 sum of D products is off by at most D 2^-24 times D of
    the largest; its roundings are independent, so a sixteenth of that is ample.  Weights:
    two bf16 parts, 2^-16."""
    c = magnitudes(counts, heads, D, False)
    got = c.run(pk, torch.float32).double().cpu().numpy()
    check_magnitudes(c, got, 2.0 ** -16, D * D * 2.0 ** -28, 0.0)


# A score over an E4M3 cache: a query element is exact down to 2^-24 of its row's largest and
# off by less than 2^-30 of that below; the sums of the products of its three parts are within
# 3 2^-20 of the largest product.  A weight is rounded to f16, half a step is 2^-11, and the
# sum is that of the weights before.

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts,heads", ROWS)
def test_query_magnitudes_over_the_whole_bf16_range_e4m3(pk, counts, heads, D):
    c = magnitudes(counts, heads, D, True)
    got = c.run(pk, torch.float32).double().cpu().numpy()
    check_magnitudes(c, got, 2.0 ** -11, 3 * 2.0 ** -20, D * 2.0 ** -30 * 448 * c.ks * c.scale)


def uneven_bound(c):
    """Of each row, what sum_j w_j |V_j| is multiplied by: the weights' 2^-11, and twice the
    scores' 2^-15 and what the smallest elements lose."""
    q = c.q.double().abs().numpy()
    most = q.max(-1, keepdims=True)
    lost = 2.0 ** -30 * most[..., 0] * (q < 2.0 ** -24 * most).sum(-1) * 448 * c.ks * c.scale
    return (2.0 ** -11 + 2 * (2.0 ** -15 + lost))[..., None]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts,heads", ROWS)
@pytest.mark.parametrize("big", [2.0 ** 9, 2.0 ** 11, 2.0 ** 13, 2.0 ** 16])
def test_a_large_query_element_over_zero_codes_costs_the_others_nothing(pk, big, counts, heads, D):
    """The others' products are at most 4.5 * 4.93 / 4, so that their sums are off by less than
    2^-15; those of elements below 2^-24 of the large one by 2^-30 of it times the keys."""
    c = Case([300, 40 + counts[1]], counts, *heads, D, True, seed=int(big) % 97)
    c.k[..., 5] = 0
    c.q[:, :, 5] = big
    c.scale *= 8
    ref, mean, _, _ = scored(c)
    got = c.run(pk, torch.float32).double().cpu().numpy()
    assert (np.abs(got - ref) <= uneven_bound(c) * mean).all()


@pytest.mark.parametrize("n", [8, 16, 20, 40])
def test_uneven_queries_beside_even_ones(pk, n):
    """Many short sequences, several a CTA, of which every other one has such an element in
    one KV head or the other."""
    B = 400
    c = Case([n + 10 + i % 23 for i in range(B)], [n] * B, 8, 2, 64, True, seed=n)
    c.k[..., 5] = 0
    for s in range(0, B, 2):
        h = s // 2 % 2
        c.q[s * n:(s + 1) * n, 4 * h:4 * h + 4, 5] = 2.0 ** (9 + s % 5)
    c.scale *= 8
    ref, mean, _, _ = scored(c)
    got = c.run(pk, torch.float32).double().cpu().numpy()
    assert (np.abs(got - ref) <= uneven_bound(c) * mean).all()


def test_one_root_over_e4m3_is_a_decode_step_for_uneven_queries(pk):
    """Both round weights to f16 and sum products in float32 (3 2^-20, and 2^-20 ample for
    the other), so that they differ by at most the sum of their errors."""
    for heads, D in (((32, 8), 128), ((8, 8), 64), ((64, 1), 128)):
        c = Case([300, 17, 1, 2000], [1, 1, 1, 1], *heads, D, True, seed=11)
        c.q[:, 0] *= 2.0 ** 14
        c.q[:, 1, 3] = 2.0 ** 12
        c.q[:, 2, ::2] *= 2.0 ** -12
        c.k[..., 3] = 0
        t = c.device()
        got = c.run(pk, torch.float32, t)
        ref = torch.empty_like(got)
        pk.paged_decode_attention(ref, t["q"], t["kc"], t["vc"], t["bt"], t["lens"], c.scale,
                                  pk.alloc_workspace(4, *heads, D, pk.FP8_E4M3), c.ks, c.vs)
        _, mean, _, top = scored(c)
        bound = (2 * 2.0 ** -11 + 2 * np.expm1(4 * 2.0 ** -20 * top))[..., None] * mean + 2.0 ** -22
        assert (np.abs((got - ref).double().cpu().numpy()) <= bound).all()


def test_an_inactive_row_of_a_padded_batch_goes_through_a_step_without_a_flag(pk):
    """Nodes, but no context: zeros from attention, a walk from verification, nothing moved."""
    c = Case([20, 30, 30], [4, 4, 4], 4, 2, 64, seed=1)
    c.lens[2] = 0
    c.check(c.run(pk, torch.float32))
    t = c.device()
    g = torch.Generator().manual_seed(0)
    prob = torch.softmax(torch.randn((12, 50), generator=g), 1).cuda()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    al, an, ot = i32(3), i32(3, 4), i32(3, 4)
    u = torch.zeros(12, device="cuda")              # every first child is accepted
    pk.kv_tree_verify(al, an, ot, prob, i32(12), t["parents"], t["starts"], u, u[:3])
    assert al[2] >= 1
    was = [t["kc"].clone(), t["vc"].clone()]
    an[0, :2], al[0] = torch.tensor([0, 3], dtype=torch.int32), 2
    an[1], al[1] = torch.tensor([0, 1, 2, 3], dtype=torch.int32), 4
    pk.kv_tree_compact(pk.CacheLayers([t["kc"]], [t["vc"]]), t["bt"], t["lens"], t["starts"], an, al)
    torch.cuda.synchronize()
    assert pk.get_device_error()[0] == 0
    bits = lambda x: x.view(torch.int16).cpu().numpy()  # noqa: E731
    k, v = R.compact(bits(was[0]), bits(was[1]), c.bt, [20, 30, 4], c.starts, an.cpu().numpy(),
                     [2, 4, 0])
    assert np.array_equal(bits(t["kc"]), k) and np.array_equal(bits(t["vc"]), v)


def test_flags_of_every_call_are_read_and_cleared(pk):
    """Each call's first bad table is seen, by the next reading only."""
    def attend(counts):
        c = Case([60 + n for n in counts], counts, 8, 2, 64, seed=1)
        t = c.device()
        t["lens"][0] = -5
        c.run(pk, t=t)

    def verify():
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        pk.kv_tree_verify(i32(1), i32(1, 3), i32(1, 3), torch.ones((3, 8), device="cuda"), i32(3),
                          i32(3) + 3, torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
                          greedy=True)

    def compact():
        k = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        pk.kv_tree_compact(pk.CacheLayers([k], [k.clone()]), i32([[0]]), i32([9]), i32([0, 4]),
                           i32([[0, 9, 9, 9]]), i32([2]))

    for call, flag in ((lambda: attend([3]), pk.DEVERR_CONTEXT_TOO_LONG),
                       (lambda: attend([40]), pk.DEVERR_CONTEXT_TOO_LONG),
                       (verify, pk.DEVERR_BAD_TREE), (compact, pk.DEVERR_BAD_TREE)):
        call()
        torch.cuda.synchronize()
        assert pk.get_device_error()[0] == flag
        assert pk.get_device_error() == (0, -1)


# A weight in one bf16 is off by at most half a step, 2^-8 of it, and their sum is that of the
# rounded ones, so that an output moves by sum_j w_j e_j (V_j - out) with |e_j| <= 2^-8, whose
# mean square over roundings of either sign is at most 2^-16 / 3 sum_j w_j^2 (V_j - out)^2; the
# output's own rounding adds at most 2^-16 / 3 out^2.  A key left out moves it by w_j (V_j - out).

def mean_square(got, ref, w2):
    """Mean square error, and what the roundings of weights and outputs may make of it."""
    return float(((got - ref) ** 2).mean()), float((2.0 ** -16 / 3 * (w2 + ref ** 2)).mean())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts,heads", [([20, 1], (8, 2)), ([40, 7], (8, 2)), ([72, 9], (16, 2))])
@pytest.mark.parametrize("ctx", [100, 1000, 6000])
def test_bf16_outputs_of_wide_trees_are_off_by_their_roundings_only(pk, ctx, counts, heads, D):
    c = Case([ctx + counts[0], 30 + counts[1]], counts, *heads, D, seed=ctx + D)
    got = c.run(pk).double().cpu().numpy()
    ref, _, scores, _ = scored(c)
    w2 = np.zeros_like(ref)
    for (t, h), (x, V) in scores.items():
        w = np.exp(x - x.max())
        w2[t, h] = (w / w.sum()) ** 2 @ (V - ref[t, h]) ** 2
    n = counts[0]                                   # the wide tree; and each of its rows alone
    err, bound = mean_square(got[:n], ref[:n], w2[:n])
    assert err <= bound
    for t, h in np.ndindex(n, heads[0]):
        # (of D columns alone: up to twice the mean)
        err, bound = mean_square(got[t, h], ref[t, h], w2[t, h])
        assert err <= 2 * bound, (t, h)
    # with one key of a row left out, up to 1000 tokens, it would not hold
    x, V = scores[n // 2, 0]
    w = np.exp(x - x.max())
    w /= w.sum()
    j = np.argsort(w)[len(w) // 2]
    lost = (ref[n // 2, 0] - w[j] * V[j]) / (1 - w[j])
    err, bound = mean_square(lost, ref[n // 2, 0], w2[n // 2, 0])
    assert err > 2 * bound or ctx > 1000


@pytest.mark.parametrize("heads,n", [((32, 8), 20), ((32, 8), 64)])
def test_bf16_outputs_of_a_full_gpu_of_long_contexts(pk, heads, n):
    Hq, Hkv, D, B, L = heads[0], heads[1], 128, 24, 3000 + n
    gen = torch.Generator(device="cuda").manual_seed(n)
    nb = -(-L // BS)
    bt = torch.randperm(B * nb, generator=gen, device="cuda").to(torch.int32).view(B, nb)
    k, v = (torch.randn((B * nb, Hkv, BS, D), generator=gen, device="cuda").to(torch.bfloat16)
            for _ in range(2))
    q = torch.randn((B * n, Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    rng = np.random.default_rng(n)
    par = np.concatenate([R.random_tree(rng, n, 3) for _ in range(B)]).astype(np.int32)
    starts = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    ws = pk.alloc_tree_workspace(B, n, Hq, Hkv, D)
    outs = []
    for _ in range(8):
        outs.append(torch.empty((B * n, Hq, D), dtype=torch.bfloat16, device="cuda"))
        pk.paged_tree_attention(outs[-1], q, k, v, bt, lens, starts, torch.from_numpy(par).cuda(), n,
                                D ** -0.5, ws)
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    G = Hq // Hkv
    for s in range(B):
        K, V = (t[bt[s].long()].double().transpose(0, 1).reshape(Hkv, -1, D)[:, :L] for t in (k, v))
        Q = q[s * n:(s + 1) * n].double().view(n, Hkv, G, D).transpose(0, 1).reshape(Hkv, n * G, D)
        mask = torch.zeros((n, L), dtype=torch.float64)
        mask[:, L - n:] = -np.inf
        for i, seen in enumerate(R.ancestors(par[s * n:(s + 1) * n])):
            mask[i, [L - n + j for j in seen]] = 0
        w = torch.softmax(Q @ K.transpose(1, 2) * D ** -0.5
                          + mask.cuda().repeat_interleave(G, 0)[None], -1)
        ref = w @ V
        # sum_j w_j^2 (V_j - out)^2
        w2 = (w * w) @ (V * V) - 2 * ((w * w) @ V) * ref + (w * w).sum(-1, keepdim=True) * ref * ref
        got = outs[0][s * n:(s + 1) * n].double().view(n, Hkv, G, D).transpose(0, 1).reshape(Hkv, n * G, D)
        for h in range(Hkv):
            err, bound = mean_square(got[h], ref[h], w2[h])
            assert err <= bound, (s, h)


@pytest.mark.parametrize("bf16,V", [(False, 4096), (False, 50001), (True, 50001)])
def test_the_drawn_token_is_that_of_the_exact_sums(pk, bf16, V):
    """The number that the last token is drawn by is, of all float32, the one that comes
    nearest to a border between two tokens: V borders beside 2^24 numbers leave about
    2^-24 / V.  Sums within 2^-44 decide it as 64 bits do; float32 sums would miss every other
    one.  One refused child, so that the sums are those of max(p - q, 0), and two, max(p - a q, 0)."""
    B = 60
    gen = torch.Generator().manual_seed(V)
    logits = torch.randn((3 * B, V), generator=gen) * 2
    dt = torch.bfloat16 if bf16 else torch.float32
    target = torch.softmax(logits, 1).to(dt)
    draft = torch.softmax(logits + torch.randn((3 * B, V), generator=gen), 1).to(dt)
    tokens = np.zeros(3 * B, dtype=np.int32)
    parents = np.tile(np.array([-1, 0, 0], dtype=np.int32), B)
    parents[5::6] = -2                              # every other sequence has one child
    starts = np.arange(0, 3 * B + 1, 3, dtype=np.int32)
    u = np.full(3 * B, 1 - 2.0 ** -24, dtype=np.float32)
    su = np.zeros(B, dtype=np.float32)
    want = np.zeros(B, dtype=np.int64)
    for s in range(B):
        p, q = (x[3 * s].double().numpy().astype(np.longdouble) for x in (target, draft))
        # tokens that are refused: the draft thinks more of them than the target does
        worse = np.nonzero(q > p * 1.01)[0]
        tokens[3 * s + 1:3 * s + 3] = worse[:2]
        R = np.maximum(p - q, 0)
        if parents[3 * s + 2] == 0:
            assert not 1.0 * q[worse[1]] * R.sum() < R[worse[1]]
            R = np.maximum(p - (1 + R.sum()) * q, 0)
        cum = np.cumsum(R)
        share = (cum / cum[-1])[:-1]
        near = share.astype(np.float32)
        gap = np.abs(near.astype(np.longdouble) - share)
        gap[(near >= 1) | (near <= 0) | (gap < 2.0 ** -41)] = 1
        i = int(np.argmin(gap))
        su[s] = near[i]
        want[s] = int(np.nonzero(cum > su[s].astype(np.longdouble) * cum[-1])[0][0])
        assert gap[i] < 2.0 ** -30
    c = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    al, an, ot = i32(B), i32(B, 3), i32(B, 3)
    pk.kv_tree_verify(al, an, ot, target.cuda(), c(tokens), c(parents), c(starts), c(u), c(su),
                      draft_probs=draft.cuda())
    assert (al == 1).all()
    assert np.array_equal(ot[:, 0].cpu().numpy(), want)


def test_caches_and_workspaces_in_host_memory_are_refused(pk):
    """They must be device memory: the others may be pinned host memory."""
    c = Case([40], [3], 4, 2, 64, seed=2)
    t = c.device()
    ws = pk.alloc_tree_workspace(1, 3, 4, 2, 64)
    for key in ("kc", "vc"):
        bad = dict(t, **{key: t[key].cpu().pin_memory()})
        with pytest.raises(ValueError, match="device memory"):
            c.run(pk, t=bad, ws=ws)
    with pytest.raises(ValueError, match="device memory"):
        c.run(pk, t=t, ws=ws.cpu().pin_memory())
    k = t["kc"].cpu().pin_memory()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError, match="device memory"):
        pk.kv_tree_compact(pk.CacheLayers([k], [k.clone().pin_memory()]), t["bt"], t["lens"],
                           t["starts"], i32(1, 3), i32(1))
