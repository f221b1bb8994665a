"""Rotary appends and latent attention on the GPU at values that the plain cases do not have:
frequencies at the ends of their range, and what must not be multiplied, in both attention kernels
and in the joining of parts."""
import numpy as np
import pytest
import torch

import latent_reference as R
from test_gpu_latent import BF, Case, check, pk, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def turns_64(freq, position):
    """position * freq as a fraction of a turn in units of 2^-64, by integers of any size."""
    unit = 1 << 400

    def arctan_of_inverse(x):
        total = term = unit // x
        k, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // k)
            k, sign = k + 2, -sign
        return total

    two_pi = 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    num, den = float(freq).as_integer_ratio()
    return (position * num * unit << 64) // (den * two_pi) % (1 << 64)


def test_frequencies_up_to_the_end_of_their_range(pk):  # noqa: F811
    """Up to 2^48, where a float's last bit is a turn of thousands, and the bits of 2 pi that count
    lie far behind its first; at and above 2^48 nothing is turned."""
    below = lambda x: float(np.nextafter(np.float32(x), np.float32(0)))  # noqa: E731
    f = [below(2.0 ** 48), 2.0 ** 47, below(2.0 ** 47), 2.0 ** 46 * 1.7, -2.0 ** 47 * 1.3, 2.0 ** 40 * 1.1,
         2.0 ** 33 * 1.9, -2.0 ** 27 * 1.01, 2.0 ** 24 * 1.5, below(2.0 ** 24), 2.0 ** 23 * 1.25, 2.0 ** 20,
         2.0 ** 48, -2.0 ** 48, 2.0 ** 90, 3.4e38]
    freq = torch.tensor(f, dtype=torch.float32)
    n, D = len(f), 2 * len(f)
    positions = torch.tensor([0, 1, 3, 1000, 8191, 123456789, 2 ** 31 + 7, -5], dtype=torch.int64)
    T = len(positions)
    q = torch.zeros((T, 1, D), dtype=BF)
    q[..., :n] = 1.0                     # turned: the cosines, then the sines
    kc, vc = (torch.zeros((1, 1, 16, D), dtype=BF, device="cuda") for _ in range(2))
    out = torch.empty((T, 1, D), dtype=BF, device="cuda")
    zero = torch.zeros((T, 1, D), dtype=BF, device="cuda")
    pk.kv_append_rotary(out, q.cuda(), zero, zero, kc, vc, torch.full((T,), -1).cuda(), positions.cuda(),
                        freq.cuda())
    want = torch.zeros((T, 1, D), dtype=torch.float64)
    for t, p in enumerate(positions.tolist()):
        for i, x in enumerate(freq.tolist()):
            a = turns_64(x, p) / 2.0 ** 64 * 2 * np.pi if abs(x) < 2.0 ** 48 else 0.0
            want[t, 0, i], want[t, 0, n + i] = np.cos(a), np.sin(a)
    # a frequency is held to 2^-63 of a turn a position; 2^-32 of a turn are cut off (part of turn_error:
    # its 2^-20 have room for more than half as much again)
    lost = positions.abs().double()[:, None, None] * 2.0 ** -63 * 2 * np.pi
    check(out, want, R.HALF_BF16 * want.abs() + R.turn_error(torch.ones_like(want)) + lost, "turns")
    assert pk.get_device_error()[0] == 0


# ------------------------------------------------------- what must not be multiplied

# both kernels (up to 64 rows a sequence, and more), both depths of their rings, contexts of one part
# and of many, nodes within a page and over the border of the pages that are weighed together
SEEN = [
    ([100, 0, 259, 31], [6, 5, 3, 1], 8, 512, 64), ([100, 0, 259, 31], [6, 5, 3, 1], 8, 256, 32),
    ([100, 0, 259, 31], [6, 5, 3, 1], 48, 256, 64), ([44, 90], [60, 9], 1, 512, 64),
    ([40, 90], [60, 9], 1, 256, 32), ([4000, 700], [41, 3], 1, 512, 32), ([4030, 9000], [40, 2], 1, 256, 64),
    ([6100, 700], [20, 3], 3, 512, 64), ([4000, 700], [60, 3], 4, 512, 64), ([5000, 700], [128, 3], 1, 256, 32),
    ([4100, 9000], [37, 2], 6, 256, 64), ([7990], [3], 100, 512, 64)]


def ancestors(par):
    seen = []
    for i in range(len(par)):
        a, mine = i, set()
        while a >= 0 and par[a] != -2:
            mine.add(a)
            a = int(par[a])
        seen.append(mine if par[i] != -2 else set())
    return seen


def row_of(c, s, pos):
    return int(c.bt[s, pos // 16]) * 16 + pos % 16


@pytest.mark.parametrize("bases,counts,H,L,rope", SEEN)
def test_what_a_node_does_not_see_does_not_reach_it(pk, bases, counts, H, L, rope):  # noqa: F811
    c = Case(bases, counts, H, L, rope, "tree", seed=H + L)
    clean = c.run(pk).cpu()
    c.check(clean)
    flat = c.cache.flatten(0, 1)
    for s, n in enumerate(c.lens):                       # the rest of each last page
        for pos in range(int(n), -(-int(n) // 16) * 16):
            flat[row_of(c, s, pos)] = float("nan") if pos % 2 else float("-inf")
    assert torch.equal(c.run(pk).cpu(), clean)
    # NaN and infinities in two drafted rows of the first sequence, one of them in the part that is turned
    n, base = int(counts[0]), int(bases[0])
    seen = ancestors(c.parents[:n])
    one, other = 1, n - 1 - n // 4
    keep = flat.clone()
    flat[row_of(c, 0, base + one), L - 9] = float("nan")
    flat[row_of(c, 0, base + other), L + 3] = float("inf")
    got = c.run(pk).cpu()
    hit = [one in seen[i] or other in seen[i] for i in range(n)]
    assert any(hit) and not all(hit)
    # (a NaN among a row's scores, or an infinite one, makes all of it NaN; -inf is a weight of zero)
    nan = torch.zeros((n, H), dtype=torch.bool)
    for i in range(n):
        nan[i] = one in seen[i]
        if other in seen[i]:
            nan[i] |= c.q[i, :, L + 3] > 0
        if not hit[i]:
            assert torch.equal(got[i], clean[i]), i
    assert torch.equal(torch.isnan(got[:n]), nan[..., None].expand(n, H, L))
    assert torch.equal(got[n:], clean[n:])
    # infinities whose scores are -inf: weight zero, but the elements themselves are NaN
    flat.copy_(keep)
    for node, col in ((one, 5), (other, L - 70)):
        flat[row_of(c, 0, base + node)] = 0.0
        flat[row_of(c, 0, base + node), col] = float("inf")
        c.q[:, :, col] = -1.0
    got = c.run(pk).cpu()
    nan = torch.zeros_like(got, dtype=torch.bool)
    for i in range(n):
        nan[i, :, 5] |= one in seen[i]
        nan[i, :, L - 70] |= other in seen[i]
    assert torch.equal(torch.isnan(got), nan)
    # the rest is as with scores that are far below the others
    for node in (one, other):
        flat[row_of(c, 0, base + node)] = 0.0
        flat[row_of(c, 0, base + node), (5 if node == one else L - 70)] = 1e30
    want, bound = R.attention(c.q, c.cache, c.bt, c.lens, c.starts, c.parents, c.scale, L)
    fine = ~nan & torch.isfinite(bound) & (bound < 1e20)
    assert fine[n:].all() and fine[~torch.tensor(hit + [False] * (len(got) - n))].all()
    over = (got.double() - want).abs() - bound
    assert (over[fine] <= 0).all()
    assert pk.get_device_error()[0] == 0


@pytest.mark.parametrize("H,L,rope", [(6, 512, 64), (9, 256, 32), (33, 512, 64), (40, 256, 64)])
def test_padding_nodes_rows_reach_nobody(pk, H, L, rope):  # noqa: F811
    c = Case([77, 2100, 10], [6, 7, 5], H, L, rope, "pads", seed=H)
    c.parents[2], c.parents[6 + 3], c.parents[6 + 4] = -2, -2, 3
    clean = c.run(pk).cpu()
    c.check(clean)
    flat = c.cache.flatten(0, 1)
    for t in np.nonzero(c.parents == -2)[0]:
        s = int(np.searchsorted(c.starts, t, side="right")) - 1
        flat[row_of(c, s, int(c.lens[s]) - int(c.starts[s + 1]) + int(t))] = float("nan")
        assert (clean[t] == 0).all()
    assert torch.equal(c.run(pk).cpu(), clean)
    assert pk.get_device_error()[0] == 0


@pytest.mark.parametrize("H,L,rope", [(16, 512, 64), (16, 256, 32), (128, 512, 64), (128, 256, 64)])
def test_nothing_of_the_call_before_is_left_in_shared_memory(pk, H, L, rope):  # noqa: F811
    """A call over NaN alone, then contexts of a few tokens, whose pages fill a part of the places."""
    bad = Case([3000] * 30, None, H, L, rope, seed=1, spread=float("nan"))
    c = Case([0, 3, 15, 16, 40, 63, 70, 130, 200], None, H, L, rope, seed=2)
    c.check(c.run(pk))
    want = c.run(pk).cpu()
    assert torch.isnan(bad.run(pk)).all()
    assert torch.equal(c.run(pk).cpu(), want)
    assert pk.get_device_error()[0] == 0


@pytest.mark.parametrize("H", [8, 100])
def test_contexts_shorter_than_their_nodes(pk, H):  # noqa: F811
    """As many of the first nodes as there is room for count; the flag tells of it."""
    c = Case([5, 40], [6, 3], H, 256, 64, seed=H)
    c.lens[0] = 4
    got = c.run(pk).cpu().double()
    assert pk.get_device_error() == (pk.DEVERR_BAD_TREE, 4)
    rows = c.cache.flatten(0, 1)[[row_of(c, 0, pos) for pos in range(4)]].double()
    for i in range(6):
        sees = rows[:i + 1]
        x = c.q[i].double() @ sees.T * c.scale
        want = torch.softmax(x, dim=1) @ sees[:, :256]
        size = torch.softmax(x, dim=1) @ sees[:, :256].abs()
        off = (c.scale * (c.q[i].double().abs() @ sees.abs().T)).amax(dim=1, keepdim=True)
        # (latent_reference.attention's bound)
        bound = 2 * R.HALF_BF16 * want.abs() + (R.HALF_BF16 + 72 * 2.0 ** -23 * off + 2.0 ** -19) * size
        assert ((got[i] - want).abs() <= bound * 1.01).all(), i


# ------------------------------------------------------------------------ captured steps

def test_a_captured_step_of_appends_and_attention(pk):  # noqa: F811
    """Two layers' latent append and attention, and a rotary append, in one graph; replayed with other
    tokens, positions, slots and lengths in the same tensors, against the same calls made one by one."""
    B, H, L, rope, NB = 3, 16, 512, 64, 60
    W = L + rope
    gen = torch.Generator().manual_seed(4)
    freq = torch.from_numpy(pk.rotary_frequencies(rope)[0]).cuda()
    weight = (1 + 0.2 * randn(gen, L)).to(BF).cuda()
    start = [randn(gen, NB, 16, W).to(BF).cuda() for _ in range(2)]
    kv0 = randn(gen, NB, 2, 16, rope).to(BF).cuda()
    bt = torch.randperm(NB, generator=gen)[:B * 20].reshape(B, 20).int().cuda()
    down, qr = torch.empty((2, B, W), dtype=BF, device="cuda"), torch.empty((2, B, H, rope), dtype=BF, device="cuda")
    q, out = torch.empty((2, B, H, W), dtype=BF, device="cuda"), torch.empty((2, B, H, L), dtype=BF, device="cuda")
    k = torch.empty((B, 2, rope), dtype=BF, device="cuda")
    qk, qo = torch.empty((B, 4, rope), dtype=BF, device="cuda"), torch.empty((B, 4, rope), dtype=BF, device="cuda")
    slots, positions = (torch.empty(B, dtype=torch.int64, device="cuda") for _ in range(2))
    lens = torch.empty(B, dtype=torch.int32, device="cuda")
    ws = pk.alloc_latent_workspace(B, 1, H, L, rope)
    caches, kc, vc = [t.clone() for t in start], kv0.clone(), kv0.clone()

    def step():
        pk.kv_append_rotary(qo, qk, k, k, kc, vc, slots, positions, freq)
        for x in range(2):
            pk.kv_latent_append(q[x][..., L:], qr[x], down[x][:, :L], down[x][:, L:], caches[x], slots, positions,
                                freq, norm_weight=weight)
            pk.paged_latent_attention(out[x], q[x], caches[x], bt, lens, 0.1, ws)

    def fill(seed, pos):
        g = torch.Generator().manual_seed(seed)
        for t in (down, qr, q, k, qk):
            t.copy_(randn(g, *t.shape).to(BF))
        p = torch.tensor(pos)
        positions.copy_(p)
        lens.copy_(p.int() + 1)
        slots.copy_(bt.cpu()[torch.arange(B), p // 16].long() * 16 + p % 16)

    fill(0, [5, 250, 100])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    results = []
    for captured in (True, False):
        for t, t0 in zip(caches + [kc, vc], start + [kv0, kv0]):
            t.copy_(t0)
        for i, pos in enumerate(([6, 251, 101], [7, 31, 318], [0, 15, 16])):
            fill(10 + i, pos)
            torch.cuda.synchronize()
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            results.append([t.cpu().clone() for t in (out, q, qo, kc, vc, *caches)])
    for a, b in zip(results[:3], results[3:]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    want, bound = R.attention(results[2][1][1], results[2][6], bt.cpu().numpy(), lens.cpu().numpy(),
                              np.arange(B + 1), None, 0.1, L)
    check(results[2][0][1], want, bound, "attention")
    assert pk.get_device_error()[0] == 0


def test_the_most_rows_of_a_sequence(pk):  # noqa: F811
    c = Case([200, 5], [128, 1], 128, 512, 64, "tree", seed=1)
    c.check(c.run(pk))
    assert pk.get_device_error()[0] == 0


@pytest.mark.parametrize("B,H,ctx", [(1, 16, 1000003), (1, 128, 700001), (90, 128, 40001), (160, 8, 30007)])
def test_long_contexts_whole_and_in_many_parts(pk, B, H, ctx):  # noqa: F811
    """Weights nearly alike over values of one sign, where what sums lose adds up; one sequence in all
    the device's parts, and more sequences than it has workers, most of them in one.  (64 bits on the
    GPU, by plain operations; latent_reference.attention's bound.)"""
    L, R_, W = 256, 32, 288
    gen = torch.Generator(device="cuda").manual_seed(B + H)
    pages = -(-ctx // 16)
    cache = torch.rand((pages + 5, 16, W), generator=gen, device="cuda").to(BF)
    # (every sequence has the same pages in another order: one copy of them is enough)
    bt = torch.stack([torch.randperm(pages - 1, generator=gen, device="cuda") for _ in range(B)]).int()
    bt = torch.cat([bt, torch.full((B, 1), pages - 1, dtype=torch.int32, device="cuda")], dim=1)
    q = (torch.randn((B, H, W), generator=gen, device="cuda") * 0.1).to(BF)
    lens = torch.full((B,), ctx, dtype=torch.int32, device="cuda")
    out = torch.empty((B, H, L), dtype=BF, device="cuda")
    ws = pk.alloc_latent_workspace(B, 1, H, L, R_)
    pk.paged_latent_attention(out, q, cache, bt, lens, 0.05, ws)
    rows = cache[:pages].flatten(0, 1)[:ctx].double()
    for b in (0, B - 1):
        x = q[b].double() @ rows.T * 0.05
        w = torch.softmax(x, dim=1)
        want = w @ rows[:, :L]
        off = 0.05 * (q[b].double().abs() @ rows.T).amax(dim=1, keepdim=True)
        rel = 72 * 2.0 ** -23 * off + (ctx / 16 + 1) * 2.0 ** -23 + 2.0 ** -20
        bound = 2 * R.HALF_BF16 * want + (R.HALF_BF16 + rel) * want
        worst = ((out[b].double() - want).abs() / want).max()
        print("B %d H %d ctx %d: %.2e of %.2e" % (B, H, ctx, worst, float((bound / want).max())))
        assert ((out[b].double() - want).abs() <= bound * 1.01).all()
    assert pk.get_device_error()[0] == 0
