"""Rotary append, latent append and latent attention on the GPU, against plain implementations in
64 bits (latent_reference.py)."""
import numpy as np
import pytest
import torch

import latent_reference as R
from tree_reference import e4m3_values, random_tree

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build_native()
    import paged_kv_cache_21_gb300 as pk
    pk.get_device_error()
    return pk


def randn(gen, *shape):
    return torch.randn(shape, generator=gen)


def check(got, want, bound, what=""):
    got = got.detach().double().cpu()
    assert torch.isfinite(got).all(), "%s: not finite" % what
    over = (got - want).abs() - bound
    assert (over <= 0).all(), "%s: %d beyond the bound, by %.3g" % (
        what, int((over > 0).sum()), float(over.max()))


# ------------------------------------------------------------------------- rotary append

ROTARY = [
    # T, Hq, Hkv, D, rotary_dim, interleaved, packed, fp8, far
    (1, 32, 8, 128, 128, False, True, False, 10),
    (1, 4, 1, 64, 16, True, False, True, 2 ** 31 - 1),
    (3, 5, 5, 64, 64, True, True, False, 2 ** 24 + 1),
    (33, 8, 2, 128, 96, False, False, True, 1000000),
    (70, 6, 3, 128, 64, True, True, True, 5000),
    (517, 7, 1, 64, 32, False, True, False, 131072),
    (1200, 32, 8, 128, 128, True, True, False, 1000000),
    (40, 0, 2, 80, 48, False, False, False, 300),
]


def rotary_inputs(T, Hq, Hkv, D, rot, packed, far, seed=0):
    gen = torch.Generator().manual_seed(seed + 7 * T + D)
    if packed:
        x = randn(gen, T, Hq + 2 * Hkv, D).to(BF)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        q, k, v = (randn(gen, T, h, D).to(BF) for h in (Hq, Hkv, Hkv))
    NB = T // 8 + 3
    slots = torch.randperm(NB * 16, generator=gen)[:T]
    positions = torch.randint(0, far, (T,), generator=gen)
    positions[0] = far - 1
    freq = (torch.tensor(10000.0, dtype=torch.float64) ** (-torch.arange(0, rot, 2) / rot)).float()
    return gen, q, k, v, NB, slots, positions, freq


def test_appends_from_pinned_host_memory_and_in_place(pk):
    """A step's own tensors in pinned host memory, as the decode entry points take them; queries
    turned where they are; negative positions, which turn the other way."""
    T, Hq, Hkv, D = 5, 4, 2, 64
    _, q, k, v, NB, slots, positions, freq = rotary_inputs(T, Hq, Hkv, D, 64, False, 900)
    positions[2] = -700
    outs = []
    for place in (lambda t: t.cuda(), lambda t: t.contiguous().pin_memory()):
        kc, vc = (torch.zeros((NB, Hkv, 16, D), dtype=BF, device="cuda") for _ in range(2))
        q_out = place(torch.empty_like(q))
        pk.kv_append_rotary(q_out, place(q), place(k), place(v), kc, vc, place(slots),
                            place(positions), place(freq))
        torch.cuda.synchronize()
        outs.append((q_out.cpu(), kc.cpu(), vc.cpu()))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    want, size = R.turn(q, positions, freq, 1.0, False)
    check(outs[0][0], want, R.HALF_BF16 * want.abs() + R.turn_error(size), "q")
    L, rope = 256, 32
    gen = torch.Generator().manual_seed(9)
    latent, kr, qr = randn(gen, T, L).to(BF), randn(gen, T, rope).to(BF), randn(gen, T, 1, rope).to(BF)
    freq = torch.from_numpy(pk.rotary_frequencies(rope)[0])
    outs = []
    for place in (lambda t: t.cuda(), lambda t: t.contiguous().pin_memory()):
        cache = torch.zeros((NB, 16, L + rope), dtype=BF, device="cuda")
        dq = place(qr.clone())
        pk.kv_latent_append(dq, dq, place(latent), place(kr), cache, place(slots), place(positions),
                            place(freq))
        torch.cuda.synchronize()
        outs.append((dq.cpu(), cache.cpu()))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    want, size = R.turn(qr, positions, freq, 1.0, False)
    check(outs[0][0], want, R.HALF_BF16 * want.abs() + R.turn_error(size), "q in place")
    assert pk.get_device_error()[0] == 0


def test_frequencies_of_any_size(pk):
    """Frequencies from 2^-140 to above a turn a position, zero and below: the angle's fraction of
    a turn in exact integers."""
    f = [0.0, 1e-42, 2.0 ** -100, 1e-20, 3e-9, 0.7, 1.0, 3.25, 6.2831855, 7.5, 1000.123, 3e7, -0.3, -9.0,
         2.0 ** -30, 12345.678]
    freq = torch.tensor(f, dtype=torch.float32)
    n, D = len(f), 2 * len(f)
    positions = torch.tensor([0, 1, 3, 1000, 123456789, 2 ** 40 + 1, -5], dtype=torch.int64)
    T = len(positions)
    q = torch.zeros((T, 1, D), dtype=BF)
    q[..., :n] = 1.0                     # turned: the cosines, then the sines
    kc, vc = (torch.zeros((1, 1, 16, D), dtype=BF, device="cuda") for _ in range(2))
    out = torch.empty((T, 1, D), dtype=BF, device="cuda")
    zero = torch.zeros((T, 1, D), dtype=BF, device="cuda")
    pk.kv_append_rotary(out, q.cuda(), zero, zero, kc, vc, torch.full((T,), -1).cuda(),
                        positions.cuda(), freq.cuda())
    # 2 pi to 220 bits, by Machin's formula; angles as fractions of a turn in 2^-64
    unit = 1 << 240

    def arctan_of_inverse(x):
        total = term = unit // x
        k, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // k)
            k, sign = k + 2, -sign
        return total

    two_pi = 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    want = torch.zeros((T, 1, D), dtype=torch.float64)
    for t, p in enumerate(positions.tolist()):
        for i, x in enumerate(freq.tolist()):
            num, den = float(x).as_integer_ratio()
            turn = (p * num * unit << 64) // (den * two_pi) % (1 << 64)
            a = torch.tensor(turn / 2.0 ** 64 * 2 * np.pi, dtype=torch.float64)
            want[t, 0, i], want[t, 0, n + i] = torch.cos(a), torch.sin(a)
    # (a frequency is held to 2^-64 of a turn a position)
    lost = positions.abs().double()[:, None, None] * 2.0 ** -64 * 2 * np.pi
    check(out, want, R.HALF_BF16 * want.abs() + R.turn_error(torch.ones_like(want)) + lost, "turns")


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,packed,fp8,far", ROTARY)
def test_rotary_append(pk, T, Hq, Hkv, D, rot, inter, packed, fp8, far):
    gen, q, k, v, NB, slots, positions, freq = rotary_inputs(T, Hq, Hkv, D, rot, packed, far)
    if T > 2:
        slots[T // 2] = -1
    mag, ks, vs = 1.25, 0.013, 0.02
    shape = (NB, Hkv, 16, D)
    if fp8:
        kc0, vc0 = (torch.randint(0, 120, shape, generator=gen, dtype=torch.uint8) for _ in range(2))
    else:
        kc0, vc0 = (randn(gen, *shape).to(BF) for _ in range(2))
    kc, vc = kc0.cuda(), vc0.cuda()
    if packed:                           # slices of one tensor on the device too
        x = torch.cat([q, k, v], dim=1).cuda()
        dq, dk, dv = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    q_out = torch.full((T, Hq + 1, D), 9.0, dtype=BF, device="cuda")[:, :Hq] if Hq else None
    pk.kv_append_rotary(q_out, dq if Hq else None, dk, dv, kc, vc, slots.cuda(), positions.cuda(),
                        freq.cuda(), interleaved=inter, magnitude=mag, k_scale=ks if fp8 else 1.0,
                        v_scale=vs if fp8 else 1.0)
    if Hq:
        want, size = R.turn(q, positions, freq, mag, inter)
        check(q_out, want, R.HALF_BF16 * want.abs() + R.turn_error(size), "q")
    k64, ksize = R.turn(k, positions, freq, mag, inter)
    live = slots >= 0
    blk, off = slots[live] // 16, slots[live] % 16
    touched = torch.zeros(shape, dtype=torch.bool)
    touched[blk, :, off] = True
    for name, got, old, x, err, scale in (("k", kc, kc0, k64, R.turn_error(ksize), ks),
                                          ("v", vc, vc0, v.double(), 0 * ksize, vs)):
        got = got.cpu()
        assert torch.equal(got[~touched], old[~touched]), name     # nothing else changes
        new = got[blk, :, off]
        if not fp8:
            check(new, x[live], R.HALF_BF16 * x[live].abs() + err[live], name)
            if name == "v":
                assert torch.equal(new, v[live])
            continue
        # a code is within half a step of the quotient: 2^-4 of a normal value, 2^-10 below
        # 2^-6; the quotient within 2^-24 of itself and the turn's error
        want = x[live] / float(np.float32(scale))
        vals = torch.from_numpy(e4m3_values())[new.long()]
        bound = want.abs() * (2.0 ** -4 + 2.0 ** -24) + 2.0 ** -10 + err[live] / scale
        assert ((vals - want.clamp(-448, 448)).abs() <= bound).all(), name
    assert pk.get_device_error()[0] == 0


def test_rotary_append_in_place_and_flags(pk):
    T, Hq, Hkv, D, rot = 37, 4, 2, 64, 64
    _, q, k, v, NB, slots, positions, freq = rotary_inputs(T, Hq, Hkv, D, rot, False, 900)
    outs = []
    for place in (False, True):
        kc, vc = (torch.zeros((NB, Hkv, 16, D), dtype=BF, device="cuda") for _ in range(2))
        dq = q.cuda()
        q_out = dq if place else torch.empty_like(dq)
        pk.kv_append_rotary(q_out, dq, k.cuda(), v.cuda(), kc, vc, slots.cuda(), positions.cuda(),
                            freq.cuda())
        outs.append((q_out.cpu(), kc.cpu(), vc.cpu()))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    # a slot behind the pool: flagged, skipped, the query turned all the same
    bad = slots.clone()
    bad[5] = NB * 16
    kc, vc = (torch.zeros((NB, Hkv, 16, D), dtype=BF, device="cuda") for _ in range(2))
    q_out = torch.empty_like(q, device="cuda")
    pk.kv_append_rotary(q_out, q.cuda(), k.cuda(), v.cuda(), kc, vc, bad.cuda(), positions.cuda(),
                        freq.cuda())
    assert pk.get_device_error() == (pk.DEVERR_SLOT_OUT_OF_RANGE, NB * 16)
    assert torch.equal(q_out.cpu(), outs[0][0])
    want = outs[0][1].clone()
    want[slots[5] // 16, :, slots[5] % 16] = 0
    assert torch.equal(kc.cpu(), want)


# ------------------------------------------------------------------------- latent append

@pytest.mark.parametrize("T,H,L,rope,inter,weighted,far", [
    (1, 128, 512, 64, False, True, 9000), (1, 1, 256, 32, True, False, 2 ** 31 - 1),
    (33, 16, 512, 64, True, True, 1000000), (130, 5, 256, 64, False, True, 50),
    (9, 0, 512, 32, False, False, 700), (700, 20, 256, 32, True, True, 131072),
    (19, 3, 1024, 128, False, True, 4000), (5, 2, 8, 16, True, True, 4000)])
def test_latent_append(pk, T, H, L, rope, inter, weighted, far):
    gen = torch.Generator().manual_seed(T + L)
    down = (randn(gen, T, L + rope + 8) * 1.5).to(BF)
    q = randn(gen, T, H, 3 * rope).to(BF)
    weight = (1 + 0.3 * randn(gen, L)).to(BF) if weighted else None
    NB = T // 8 + 2
    cache0 = randn(gen, NB, 16, L + rope).to(BF)
    slots = torch.randperm(NB * 16, generator=gen)[:T]
    if T > 3:
        slots[1] = -1
        down[2, :L] = 0.0                # a vector of zeros stays one
    positions = torch.randint(0, far, (T,), generator=gen)
    positions[-1] = far - 1
    freq = torch.from_numpy(pk.rotary_frequencies(rope, 10000.0)[0])
    mag, eps = 0.9, 1e-5
    cache, ddown, dq = cache0.cuda(), down.cuda(), q.cuda()
    full = torch.full((T, H, L + rope), 3.0, dtype=BF, device="cuda")
    pk.kv_latent_append(full[..., L:] if H else None, dq[..., rope:2 * rope] if H else None,
                        ddown[:, :L], ddown[:, L:L + rope], cache, slots.cuda(), positions.cuda(),
                        freq.cuda(), norm_weight=weight.cuda() if weighted else None, eps=eps,
                        interleaved=inter, magnitude=mag)
    if H:
        want, size = R.turn(q[..., rope:2 * rope], positions, freq, mag, inter)
        check(full[..., L:], want, R.HALF_BF16 * want.abs() + R.turn_error(size), "q")
        assert (full[..., :L] == 3.0).all()
    live = slots >= 0
    got = cache.cpu()
    want, size = R.turn(down[:, None, L:L + rope], positions, freq, mag, inter)
    new = got.flatten(0, 1)[slots[live]]
    check(new[:, L:], want[live, 0], (R.HALF_BF16 * want.abs() + R.turn_error(size))[live, 0], "key")
    # the sum of squares and its root, quotient and two products in float32: L / 32 + 5 additions
    # and five more roundings of 2^-24
    x = R.norm(down[:, :L], weight, eps)[live]
    check(new[:, :L], x, x.abs() * (R.HALF_BF16 + (L / 32 + 10) * 2.0 ** -24), "latent")
    if not weighted:
        assert torch.equal(new[:, :L], down[live, :L])
    rest = torch.ones(NB * 16, dtype=torch.bool)
    rest[slots[live]] = False
    assert torch.equal(got.flatten(0, 1)[rest], cache0.flatten(0, 1)[rest])
    assert pk.get_device_error()[0] == 0


# ---------------------------------------------------------------------- latent attention

class Case:
    """Sequences of `bases` committed tokens and trees of `counts` nodes (None: one token each,
    without tables); kind "chain", "tree" or "pads"."""

    def __init__(self, bases, counts, H, L, rope, kind="chain", seed=0, scale=None, spread=1.0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.single = counts is None
        counts = np.ones(len(bases), dtype=int) if counts is None else np.asarray(counts)
        self.H, self.L, self.W = H, L, L + rope
        self.lens = np.asarray(bases) + counts
        self.starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.total, self.max_nodes = int(self.starts[-1]), int(counts.max())
        need = -(-self.lens // 16)
        self.NB = int(need.sum()) + 3
        perm = rng.permutation(self.NB)
        self.bt = np.full((len(bases), max(1, int(need.max())) + 1), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            self.bt[s, :n] = perm[at:at + n]
            at += n
        self.parents = None
        if kind != "chain":
            self.parents = np.concatenate(
                [random_tree(rng, int(n), 3, 0.2 if kind == "pads" else 0.0) for n in counts] +
                [np.zeros(0, dtype=np.int32)]).astype(np.int32)
        self.q = (randn(gen, self.total, H, self.W) * 1.5).to(BF)
        self.cache = (randn(gen, self.NB, 16, self.W) * spread).to(BF)
        self.scale = 2.0 * self.W ** -0.5 if scale is None else scale

    def run(self, pk, ws=None, stream=None, out=None):
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        if out is None:
            out = torch.full((self.total, self.H, self.L), 5.0, dtype=BF, device="cuda")
        if ws is None:
            ws = pk.alloc_latent_workspace(len(self.lens), self.max_nodes, self.H, self.L,
                                           self.W - self.L)
            ws.fill_(255)                # NaN wherever it is read before it is written
        pk.paged_latent_attention(
            out, self.q.cuda(), self.cache.cuda(), i32(self.bt), i32(self.lens), self.scale, ws,
            node_starts=None if self.single else i32(self.starts),
            parents=None if self.parents is None else i32(self.parents),
            max_nodes=self.max_nodes, stream=stream)
        torch.cuda.synchronize()
        return out

    def check(self, out):
        want, bound = R.attention(self.q, self.cache, self.bt, self.lens, self.starts, self.parents,
                                  self.scale, self.L)
        check(out, want, bound, "attention")


SIZES = [
    # bases, counts, heads, latent, rope, kind
    ([127], None, 16, 512, 64, "chain"),
    ([0], None, 1, 256, 32, "chain"),
    ([0, 1, 14, 15, 16, 17, 126, 127, 128, 129], None, 16, 512, 64, "chain"),
    ([300, 5, 1000], None, 128, 512, 64, "chain"),
    ([300, 5, 1000], None, 128, 256, 64, "chain"),
    ([511, 40], None, 65, 512, 32, "chain"),
    ([63, 64, 65], None, 63, 256, 32, "chain"),
    ([9000], None, 5, 512, 64, "chain"),
    ([2500, 40, 2047, 3], None, 40, 256, 32, "chain"),
    ([100, 0, 259], [3, 2, 1], 16, 512, 64, "chain"),
    ([200, 33], [4, 1], 128, 512, 64, "chain"),
    ([90], [128], 1, 256, 64, "chain"),
    ([30, 700], [50, 9], 7, 512, 64, "tree"),
    ([0, 16, 250], [12, 33, 1], 20, 256, 32, "tree"),
    ([77, 130, 10], [20, 6, 5], 33, 512, 64, "pads"),
    ([64], [128], 5, 512, 64, "tree"),
    ([1500], [40], 128, 512, 64, "tree"),
    # contexts that many workers share: parts by the dozen, with rows for either kernel
    ([20000], None, 16, 512, 64, "chain"),
    ([12000], [2], 100, 512, 64, "chain"),
    ([7000, 3000], [3, 1], 60, 256, 32, "tree"),
]


@pytest.mark.parametrize("bases,counts,H,L,rope,kind", SIZES)
def test_latent_attention(pk, bases, counts, H, L, rope, kind):
    c = Case(bases, counts, H, L, rope, kind, seed=len(bases) + H)
    c.check(c.run(pk))
    assert pk.get_device_error()[0] == 0


def test_latent_attention_many_sequences(pk):
    """More sequences than the device runs at once, most of them short."""
    rng = np.random.default_rng(5)
    c = Case(rng.integers(0, 90, size=333), None, 16, 256, 32, seed=5)
    c.check(c.run(pk))
    c = Case(rng.integers(0, 60, size=170), rng.integers(0, 4, size=170), 64, 512, 64, "tree", seed=6)
    c.check(c.run(pk))
    assert pk.get_device_error()[0] == 0


def test_latent_attention_rising_scores(pk):
    """References that move many times: a token's score grows along the context, by 2^8 and more
    between chunks, and falls again."""
    c = Case([1400, 700], None, 32, 512, 64, seed=3, spread=0.05)
    u = torch.randn(c.W, generator=torch.Generator().manual_seed(1))
    u /= u.norm()
    for s, n in enumerate(c.lens):
        rise = torch.linspace(0, 1, int(n)) if s == 0 else torch.linspace(1, 0, int(n))
        flat = c.cache.flatten(0, 1)
        slots = torch.as_tensor(c.bt[s, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16)
        flat[slots] = (flat[slots].float() + rise[:, None] * u * 40).to(BF)
    c.q = (c.q.float() + u * 25).to(BF)
    c.scale = 0.5
    c.check(c.run(pk))


def test_latent_attention_does_not_read_what_a_node_does_not_see(pk):
    """Infinities and NaN behind the contexts, and at drafted positions for the nodes that do not
    see them."""
    c = Case([100, 0, 259, 31], [6, 5, 3, 1], 48, 512, 64, "tree", seed=9)
    clean = c.run(pk).cpu()
    c.check(clean)
    flat = c.cache.flatten(0, 1)
    for s, n in enumerate(c.lens):                       # the rest of each last page
        for pos in range(int(n), -(-int(n) // 16) * 16):
            flat[int(c.bt[s, pos // 16]) * 16 + pos % 16] = float("nan") if pos % 2 else float("inf")
    dirty = c.run(pk).cpu()
    assert torch.equal(dirty, clean)
    # node 2 of the first sequence: NaN in its row, seen by itself and its descendants
    par = c.parents
    base = int(c.lens[0] - 6)
    flat[int(c.bt[0, (base + 2) // 16]) * 16 + (base + 2) % 16, 7] = float("nan")
    got = c.run(pk).cpu()
    sees = [False] * 6
    for i in range(6):
        a = i
        while a >= 0:
            sees[i] = sees[i] or a == 2
            a = int(par[a])
    assert any(sees) and not all(sees)
    for i in range(6):
        if sees[i]:
            assert torch.isnan(got[i]).all()
        else:
            assert torch.equal(got[i], clean[i])
    assert torch.equal(got[6:], clean[6:])
    # an infinity whose score is -inf: weight zero, but the element itself is NaN
    c.cache.flatten(0, 1)[int(c.bt[0, (base + 2) // 16]) * 16 + (base + 2) % 16] = 0.0
    c.cache.flatten(0, 1)[int(c.bt[0, (base + 2) // 16]) * 16 + (base + 2) % 16, 300] = float("inf")
    c.q[:, :, 300] = -1.0
    got = c.run(pk).cpu()
    for i in range(6):
        nan = torch.isnan(got[i])
        want = torch.zeros_like(nan)
        if sees[i]:
            want[:, 300] = True
        assert torch.equal(nan, want), i


def test_latent_attention_rows_without_positions(pk):
    """Sequences without a context, without nodes, and rows behind the last node."""
    c = Case([50, 0, 20], [2, 0, 3], 24, 256, 64, seed=4)
    c.lens[2] = 0
    out = torch.full((c.total + 2, c.H, c.L), 5.0, dtype=BF, device="cuda")
    c.q = torch.cat([c.q, c.q[:2]])
    full, c.total = c.total, c.total + 2
    got = c.run(pk, out=out)
    c.total = full
    c.q = c.q[:full]
    c.check(got[:full])
    assert (got[2:5] == 0).all() and (got[full:] == 5.0).all()
    # a committed row of -inf scores alone has no softmax
    c = Case([0], None, 3, 256, 32, seed=2)
    c.cache[:] = 0.0
    c.cache[..., 1] = float("inf")
    c.q[:] = 0.0
    c.q[..., 1] = -1.0
    assert torch.isnan(c.run(pk)).all()


def test_latent_attention_flags(pk):
    c = Case([100, 60], [2, 2], 16, 512, 64, seed=8)
    good = c.run(pk).cpu()
    c.bt[0, 2] = c.NB
    got = c.run(pk).cpu()
    assert pk.get_device_error() == (pk.DEVERR_BLOCK_OUT_OF_RANGE, c.NB)
    assert torch.equal(got[2:], good[2:])
    c.bt[0, 2] = 0
    c.lens[0] = c.bt.shape[1] * 16 + 1
    c.bt[0, :] = 1
    c.run(pk)
    assert pk.get_device_error() == (pk.DEVERR_CONTEXT_TOO_LONG, int(c.lens[0]))
    c = Case([100, 60], [2, 2], 16, 512, 64, seed=8)
    c.starts = np.array([0, 9, 4], dtype=np.int32)
    out = torch.full((4, 16, 512), 5.0, dtype=BF, device="cuda")
    c.run(pk, out=out)
    assert pk.get_device_error()[0] == pk.DEVERR_BAD_TREE
    c = Case([100, 60], [2, 2], 16, 512, 64, "tree", seed=8)
    c.parents[1] = 7
    c.run(pk)
    assert pk.get_device_error() == (pk.DEVERR_BAD_TREE, 7)
    c.parents[1] = -1                    # what a bad parent counts as
    c.check(c.run(pk))
    assert pk.get_device_error()[0] == 0


def test_latent_attention_repeats_and_streams(pk):
    """The same bits again, whatever the blocks, on another stream, from a captured graph, and two
    calls at once with a workspace each."""
    c = Case([700, 3000, 5], [3, 1, 2], 64, 512, 64, "tree", seed=12)
    first = c.run(pk).cpu()
    c.check(first)
    assert torch.equal(c.run(pk).cpu(), first)
    perm = np.random.default_rng(1).permutation(c.NB)
    moved = torch.empty_like(c.cache)
    moved[torch.from_numpy(perm)] = c.cache
    keep = c.cache, c.bt.copy()
    c.cache, c.bt = moved, np.where(c.bt >= 0, perm[np.maximum(c.bt, 0)], -1).astype(np.int32)
    assert torch.equal(c.run(pk).cpu(), first)
    c.cache, c.bt = keep
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    args = (c.q.cuda(), c.cache.cuda(), i32(c.bt), i32(c.lens), c.scale)
    tables = dict(node_starts=i32(c.starts), parents=i32(c.parents), max_nodes=c.max_nodes)
    outs = [torch.empty((c.total, c.H, c.L), dtype=BF, device="cuda") for _ in range(3)]
    wss = [pk.alloc_latent_workspace(3, 3, c.H, c.L, 64) for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, w in ((s1, outs[0], wss[0]), (s2, outs[1], wss[1])):
            pk.paged_latent_attention(o, *args, w, stream=s, **tables)
    torch.cuda.synchronize()
    assert torch.equal(outs[0].cpu(), first) and torch.equal(outs[1].cpu(), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.paged_latent_attention(outs[2], *args, wss[2], **tables)
    outs[2].zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[2].cpu(), first)


@pytest.mark.parametrize("H", [16, 128])
def test_latent_attention_gives_up_a_wait_that_runs_out(pk, H):
    """The test hook: a wait of the kernel's scores runs out, the flag says so, and the next call
    is right."""
    c = Case([700, 90], None, H, 512, 64, seed=H)
    pk.set_pipeline_stall(1000)
    try:
        c.run(pk)
    finally:
        pk.set_pipeline_stall(0)
    assert pk.get_device_error()[0] & pk.DEVERR_PIPELINE_TIMEOUT
    c.check(c.run(pk))
    assert pk.get_device_error()[0] == 0


@pytest.mark.parametrize("H,n", [(16, 1), (64, 2)])
def test_latent_attention_large_and_tiny_scores(pk, H, n):
    """Scores above 2^21, whose products are rounded by 2^-3 and more, and weights that all but
    one lose: the weight of the largest is one whatever its rounding."""
    c = Case([300], [n], H, 256, 64, seed=7)
    flat = c.cache.flatten(0, 1)
    c.q = torch.full_like(c.q, 64.0)
    flat[:] = torch.randn(flat.shape, generator=torch.Generator().manual_seed(1)).to(BF) * 0.01
    hot = 123
    flat[int(c.bt[0, hot // 16]) * 16 + hot % 16] = 500.0
    c.scale = 3.0                        # 64 * 500 * 320 * 3 = 3.1e7 for the one
    out = c.run(pk).cpu()
    assert (out == 500.0).all()


# ------------------------------------------------------------------------- used together

def test_a_run_of_steps_over_latent_caches(pk):
    """Sequences with a fork, two layers: drafted steps as a program makes them (allocator, copies
    of shared blocks, append, attention, verification, compaction, truncation), the caches and the
    attention against a plain list of rows a sequence."""
    L, rope, H, NB, V = 256, 32, 12, 40, 50
    W = L + rope
    gen = torch.Generator().manual_seed(0)
    rng = np.random.default_rng(0)
    freq, mag = pk.rotary_frequencies(rope, 10000.0, scaling="linear", factor=4.0)
    freq = torch.from_numpy(freq)
    alloc = pk.BlockAllocator(NB, 1, W // 2)
    caches = [torch.zeros((NB, 16, W), dtype=BF, device="cuda") for _ in range(2)]
    layers = pk.CacheLayers(caches)
    weight = (1 + 0.2 * randn(gen, L)).to(BF)
    alloc.add(0, 0)
    rows = {0: [[], []]}                 # each sequence's rows, by layer, as the cache should hold them
    ids = [0]
    ws = pk.alloc_latent_workspace(3, 6, H, L, rope)
    for step in range(7):
        if step == 3:                    # a fork inside a block
            alloc.fork(0, 1, len(rows[0][0]))
            rows[1] = [list(rows[0][0]), list(rows[0][1])]
            ids = [0, 1]
        counts = rng.integers(1, 7, size=len(ids)) if step else np.array([6])
        slots, bt, lens, starts, (src, dst) = alloc.tree_step(ids, counts, max_blocks=8)
        base = lens - counts
        par = np.concatenate([random_tree(rng, int(n), 2) for n in counts])
        if len(src):
            for cache in caches:
                pk.kv_copy_blocks(cache, None, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda())
        depth = np.zeros(len(par), dtype=np.int64)
        for s, n in enumerate(counts):
            for i in range(int(n)):
                p = par[starts[s] + i]
                depth[starts[s] + i] = 0 if p < 0 else depth[starts[s] + p] + 1
        positions = torch.from_numpy(np.repeat(base, counts).astype(np.int64) + depth)
        T = int(starts[-1])
        dev = [torch.from_numpy(a).cuda() for a in (bt, lens, starts, par)]
        new = []
        for cache in caches:
            down = randn(gen, T, W).to(BF)
            qr = randn(gen, T, H, rope).to(BF)
            q = randn(gen, T, H, W).to(BF).cuda()
            pk.kv_latent_append(q[..., L:], qr.cuda(), down[:, :L].cuda(), down[:, L:].cuda(), cache,
                                torch.from_numpy(slots).cuda(), positions.cuda(), freq.cuda(),
                                norm_weight=weight.cuda(), magnitude=mag)
            out = torch.empty((T, H, L), dtype=BF, device="cuda")
            pk.paged_latent_attention(out, q, cache, dev[0], dev[1], 0.1, ws, node_starts=dev[2],
                                      parents=dev[3], max_nodes=6)
            # what the cache holds of the new rows, checked against the formulas
            held = cache.cpu().flatten(0, 1)[torch.from_numpy(slots)]
            k64, size = R.turn(down[:, None, L:], positions, freq, mag, False)
            check(held[:, L:], k64[:, 0], (R.HALF_BF16 * k64.abs() + R.turn_error(size))[:, 0], "key")
            x = R.norm(down[:, :L], weight, 1e-6)
            check(held[:, :L], x, x.abs() * (R.HALF_BF16 + (L / 32 + 10) * 2.0 ** -24), "latent")
            new.append(held)
            want, bound = R.attention(q.cpu(), cache.cpu(), bt, lens, starts, par, 0.1, L)
            check(out, want, bound, "attention")
        target = torch.randn((T, V), generator=gen)
        tokens = torch.randint(0, V, (T,), generator=gen, dtype=torch.int32)
        best = target.argmax(dim=1)
        for s, n in enumerate(counts):   # half of the children are what the target wants
            for i in range(1, int(n)):
                if rng.random() < 0.5 and par[starts[s] + i] >= 0:
                    tokens[starts[s] + i] = best[starts[s] + par[starts[s] + i]]
        accept_lens = torch.empty(len(ids), dtype=torch.int32, device="cuda")
        nodes, toks = (torch.empty((len(ids), 6), dtype=torch.int32, device="cuda") for _ in range(2))
        pk.kv_tree_verify(accept_lens, nodes, toks, target.cuda(), tokens.cuda(), dev[3], dev[2],
                          greedy=True)
        pk.kv_tree_compact(layers, dev[0], dev[1], dev[2], nodes, accept_lens)
        took, path = accept_lens.cpu().numpy(), nodes.cpu().numpy()
        alloc.truncate(ids, base + took)
        for s, sid in enumerate(ids):
            for layer in range(2):
                rows[sid][layer] += [new[layer][starts[s] + int(i)] for i in path[s, :took[s]]]
        for sid in ids:                  # the sequences' rows, through their tables
            n, blocks = alloc.info(sid)
            assert n == len(rows[sid][0])
            for layer in range(2):
                held = caches[layer].cpu()[torch.from_numpy(blocks).long()].flatten(0, 1)[:n]
                assert torch.equal(held, torch.stack(rows[sid][layer])), (step, sid, layer)
    assert alloc.trace([0])[0]["cache_bytes"] == len(alloc.info(0)[1]) * 16 * W * 2
    assert pk.get_device_error()[0] == 0


def test_rotary_append_then_decode(pk):
    """A decode step whose keys and queries are turned on the way: kv_append_rotary, then
    paged_decode_attention, against the turned vectors in 64 bits."""
    gen = torch.Generator().manual_seed(3)
    B, Hq, Hkv, D, N = 3, 8, 2, 64, 70
    freq, mag = pk.rotary_frequencies(D, 10000.0, scaling="parts", factor=4.0, original_len=64.0)
    freq = torch.from_numpy(freq)
    NB = 20
    kc, vc = (torch.zeros((NB, Hkv, 16, D), dtype=BF, device="cuda") for _ in range(2))
    alloc = pk.BlockAllocator(NB, Hkv, D)
    keys, vals = [[] for _ in range(B)], [[] for _ in range(B)]
    for s in range(B):
        alloc.add(s, 0)
    ws = pk.alloc_workspace(B, Hq, Hkv, D)
    for pos in range(N):
        x = randn(gen, B, Hq + 2 * Hkv, D).to(BF)
        slots, bt, lens, _ = alloc.step(list(range(B)), max_blocks=8)
        p = torch.full((B,), pos, dtype=torch.int64)
        d = x.cuda()
        q = torch.empty((B, Hq, D), dtype=BF, device="cuda")
        pk.kv_append_rotary(q, d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], kc, vc,
                            torch.from_numpy(slots).cuda(), p.cuda(), freq.cuda(), magnitude=mag)
        k64, _ = R.turn(x[:, Hq:Hq + Hkv], p, freq, mag, False)
        for s in range(B):
            keys[s].append(k64[s])
            vals[s].append(x[s, Hq + Hkv:].double())
    out, early = (torch.empty((B, Hq, D), dtype=torch.float32, device="cuda") for _ in range(2))
    tables = torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda()
    pk.paged_decode_attention(out, q, kc, vc, *tables, D ** -0.5, ws)
    # the last append again and, directly behind it, the step that reads the cache early
    torch.cuda.synchronize()
    slots, p = torch.from_numpy(slots).cuda(), p.cuda()
    kc2, vc2 = kc.clone(), vc.clone()
    freq = freq.cuda()
    for cache in (kc2, vc2):
        for s in range(B):
            cache[int(slots[s]) // 16, :, int(slots[s]) % 16] = 7.0
    torch.cuda.synchronize()
    q2 = torch.empty_like(q)
    pk.kv_append_rotary(q2, d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], kc2, vc2, slots, p, freq,
                        magnitude=mag)
    pk.paged_decode(early, q2, kc2, vc2, *tables, D ** -0.5, ws, early_inputs=True)
    assert torch.equal(early.cpu(), out.cpu()) and torch.equal(kc2.cpu(), kc.cpu())
    p, freq = p.cpu(), freq.cpu()
    q64, _ = R.turn(x[:, :Hq], p, freq, mag, False)
    G = Hq // Hkv
    for s in range(B):
        k, v = torch.stack(keys[s]), torch.stack(vals[s])
        for h in range(Hq):
            w0 = q64[s, h] @ k[:, h // G].T * D ** -0.5
            w = torch.softmax(w0, dim=0)
            # a score is off by the roundings of the turned query and key, 2^-8 each, so a weight
            # by twice that; the weights and sums of the decode kernel by 2^-8 more
            off = (q64[s, h].abs() @ k[:, h // G].abs().T).max() * D ** -0.5 * 2.0 ** -7
            size = w @ v[:, h // G].abs()
            assert ((out[s, h].cpu().double() - w @ v[:, h // G]).abs()
                    <= (torch.exp(2 * off) - 1 + 2.0 ** -8) * size).all()


@pytest.mark.parametrize("B,H,nodes", [(32, 16, 0), (33, 16, 0), (512, 8, 0), (513, 8, 2), (1100, 4, 0),
                                       (600, 70, 2)])
def test_latent_attention_shares_of_any_batch(pk, B, H, nodes):
    """The work is cut by one warp, by all of a CTA, or by it in turns, as the batch has it; some
    sequences have no context, and some no nodes."""
    rng = np.random.default_rng(B)
    counts = None if nodes == 0 else rng.integers(0, nodes + 1, size=B)
    c = Case(rng.integers(0, 40, size=B), counts, H, 256, 32, seed=B)
    c.lens[3 % B] = 0 if counts is None else c.lens[3 % B]
    c.lens[B - 1] = 0 if counts is None else c.lens[B - 1]
    c.check(c.run(pk))
    assert pk.get_device_error()[0] == 0


def test_latent_attention_one_long_among_many_empty(pk):
    """Behind a thousand sequences without a context, the last one's pages are shared out."""
    c = Case(np.concatenate([np.zeros(1030, dtype=int), [2500]]), None, 16, 256, 32, seed=3)
    c.lens[:1030] = 0
    c.check(c.run(pk))
    assert pk.get_device_error()[0] == 0


@pytest.mark.parametrize("H", [16, 128])
def test_blocks_far_into_a_large_cache(pk, H):
    """Blocks whose bytes and elements are behind 2^32, appended to and attended over."""
    L, rope = 512, 64
    W = L + rope
    NB = 2 ** 32 // (16 * W) + 40                    # 8.6 GB, of which only the last pages are used
    cache = torch.empty((NB, 16, W), dtype=BF, device="cuda")
    c = Case([150], None, H, L, rope, seed=H)
    n = int(c.lens[0])
    blocks = NB - 1 - np.arange(-(-n // 16)) * 2
    gen = torch.Generator().manual_seed(1)
    rows = randn(gen, n, W).to(BF)
    slots = torch.from_numpy(blocks[np.arange(n) // 16] * 16 + np.arange(n) % 16)
    assert int(slots.max()) * W > 2 ** 32
    still = torch.zeros(n, dtype=torch.int64)        # (position 0 turns nothing)
    pk.kv_latent_append(None, None, rows[:, :L].cuda(), rows[:, L:].cuda(), cache, slots.cuda(),
                        still.cuda(), torch.ones(rope // 2).cuda())
    used = torch.from_numpy(blocks).cuda()
    small = cache[used].cpu()
    assert torch.equal(small.flatten(0, 1)[:n], rows)
    bt = torch.from_numpy(blocks.astype(np.int32))[None].cuda()
    out = torch.empty((1, H, L), dtype=BF, device="cuda")
    ws = pk.alloc_latent_workspace(1, 1, H, L, rope)
    pk.paged_latent_attention(out, c.q.cuda(), cache, bt, torch.tensor([n], dtype=torch.int32).cuda(),
                              c.scale, ws)
    want, bound = R.attention(c.q, small, np.arange(len(blocks))[None], [n], [0, 1], None, c.scale, L)
    check(out, want, bound, "attention")
    assert pk.get_device_error()[0] == 0


def test_latent_attention_tables_in_pinned_memory(pk):
    for H in (9, 100):
        c = Case([90, 0, 259], [4, 3, 1], H, 256, 64, "tree", seed=H)
        first = c.run(pk).cpu()
        pin = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).pin_memory()  # noqa: E731
        out = torch.empty((c.total, H, 256), dtype=BF, device="cuda")
        ws = pk.alloc_latent_workspace(3, 4, H, 256, 64)
        tables = pin(c.bt), pin(c.lens), pin(c.starts), pin(c.parents)
        pk.paged_latent_attention(out, c.q.cuda(), c.cache.cuda(), tables[0], tables[1], c.scale, ws,
                                  node_starts=tables[2], parents=tables[3], max_nodes=4)
        assert torch.equal(out.cpu(), first)


def test_calls_of_both_kernels_share_a_workspace_one_after_the_other(pk):
    """Back to back on a stream, each launched while the one before drains: few rows, many rows,
    split and whole, with the workspace of the largest."""
    cases = [Case([5000], None, 16, 512, 64, seed=1), Case([3000, 40], [3, 2], 50, 512, 64, seed=2),
             Case([20], None, 128, 512, 64, seed=3), Case([700, 900], [1, 2], 20, 512, 64, seed=4)]
    want = [c.run(pk).cpu() for c in cases]
    ws = pk.alloc_latent_workspace(2, 128, 128, 512, 64)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    calls = []
    for c in cases:
        calls.append(((c.q.cuda(), c.cache.cuda(), i32(c.bt), i32(c.lens), c.scale, ws),
                      dict(node_starts=None if c.single else i32(c.starts), max_nodes=c.max_nodes)))
    outs = [[torch.empty_like(w, device="cuda") for w in want] for _ in range(6)]
    torch.cuda.synchronize()
    for r in outs:
        for out, (args, kw) in zip(r, calls):
            pk.paged_latent_attention(out, *args, **kw)
    torch.cuda.synchronize()
    for r in outs:
        for out, w in zip(r, want):
            assert torch.equal(out.cpu(), w)


@pytest.mark.parametrize("H,n", [(16, 1), (40, 3)])
@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_latent_attention_scales_of_any_sign(pk, H, n, scale):
    c = Case([400, 30], [n, 1], H, 256, 64, "tree", seed=H, scale=scale)
    c.check(c.run(pk))


@pytest.mark.parametrize("H,n", [(16, 1), (40, 3)])
def test_latent_attention_rows_do_not_reach_each_other(pk, H, n):
    """NaN, infinities and the largest values in some queries change no other row's bits, in
    sequences of one part and of several."""
    c = Case([4000, 300, 30], [n, n, 1], H, 512, 64, seed=H)
    clean = c.run(pk).cpu()
    c.check(clean)
    bad = {(0, 1): float("nan"), (0, H - 1): float("inf"), (n, 5): -float("inf"),
           (n, 7): 3.3e38, (2 * n, 0): float("nan")}
    for (t, h), x in bad.items():
        c.q[t, h, 3] = x
    got = c.run(pk).cpu()
    for (t, h), x in bad.items():
        if x != x:
            assert torch.isnan(got[t, h]).all()
        got[t, h] = clean[t, h]
    assert torch.equal(got, clean)
    assert pk.get_device_error()[0] == 0


def test_no_tokens_and_no_sequences(pk):
    cache = torch.full((4, 16, 288), 2.0, dtype=BF, device="cuda")
    kc = torch.full((4, 2, 16, 64), 2.0, dtype=BF, device="cuda")
    e = lambda *s, t=BF: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    none = e(0, t=torch.int64)
    pk.kv_append_rotary(e(0, 4, 64), e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), kc, kc.clone(), none, none,
                        e(32, t=torch.float32))
    pk.kv_latent_append(e(0, 4, 32), e(0, 4, 32), e(0, 256), e(0, 32), cache, none, none,
                        e(16, t=torch.float32))
    ws = pk.alloc_latent_workspace(0, 1, 4, 256, 32)
    i32 = torch.int32
    pk.paged_latent_attention(e(0, 4, 256), e(0, 4, 288), cache, e(0, 3, t=i32), e(0, t=i32), 0.1, ws)
    torch.cuda.synchronize()
    assert (cache == 2.0).all() and (kc == 2.0).all()
    # nodes without sequences' contexts, sequences without nodes
    out = torch.full((1, 4, 256), 5.0, dtype=BF, device="cuda")
    starts = torch.tensor([0, 0, 0], dtype=i32, device="cuda")
    bt = torch.zeros((2, 2), dtype=i32, device="cuda")
    pk.paged_latent_attention(out, torch.ones((1, 4, 288), dtype=BF, device="cuda"), cache, bt,
                              torch.tensor([20, 0], dtype=i32, device="cuda"), 0.1, ws,
                              node_starts=starts)
    assert (out == 5.0).all()
    assert pk.get_device_error()[0] == 0
