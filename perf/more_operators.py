"""Cases, plain forms and exact values of the operators around rotary positions and latent caches:
rotation of queries and keys on their way into the paged cache, the append of a normalised latent
vector with its rotary key, and attention over the latent cache (absorbed form).  ``run`` is the
plain form while ``own`` is false and the library's call while it is true."""
import math

import numpy as np
import torch

own = False

BLOCK = 16
EPS = 1e-6


def _pk():
    import paged_kv_cache_21_gb300 as pk
    return pk


# ---------------------------------------------------------------------- cases

def _rotary(name, T, Hq, Hkv, D, rot, inter, chunk, far, theta, factor, packed=True, fp8=False):
    """T tokens, `chunk` consecutive positions a sequence, positions up to `far`."""
    c = {"op": "rotary", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "inter": inter,
         "chunk": chunk, "far": far, "theta": theta, "factor": factor, "packed": packed,
         "fp8": fp8}
    if name:
        c["name"] = name
    return c


def _lappend(name, T, H, L, R, inter, norm, chunk, far, factor):
    c = {"op": "latent_append", "T": T, "H": H, "L": L, "R": R, "inter": inter, "norm": norm,
         "chunk": chunk, "far": far, "factor": factor}
    if name:
        c["name"] = name
    return c


def _latent(name, B, H, L, R, ctx_lo, ctx_hi, nodes_lo, nodes_hi, width):
    """width 0: one token a sequence, without tree tables; 1: chains of drafted tokens; above:
    trees."""
    c = {"op": "latent", "B": B, "H": H, "L": L, "R": R, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
         "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "width": width}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the next token of one request: the latency of the call
        _rotary("rotary 1 32q/8kv", 1, 32, 8, 128, 128, False, 1, 9000, 500000.0, 8.0),
        # a decode step of a large batch over an E4M3 cache, part of the head rotated, adjacent
        # elements paired
        _rotary("rotary 256 32q/8kv e4m3 64 of 128", 256, 32, 8, 128, 64, True, 1, 100000, 10000.0,
                1.0, fp8=True),
        # a chunk of prompts, far into a scaled context
        _rotary("rotary 8192 32q/8kv", 8192, 32, 8, 128, 128, False, 512, 1000000, 500000.0, 32.0),
        # a decode step of a batch, all heads of a layer on this device
        _lappend("latent append 32 128h", 32, 128, 512, 64, True, True, 1, 8192, 1.0),
        # a chunk of prompts, the heads shared out over eight devices
        _lappend("latent append 8192 16h", 8192, 16, 512, 64, False, True, 512, 131072, 40.0),
        # one request, a short context: the latency of the call
        _latent("latent 1x128 16h", 1, 16, 512, 64, 128, 128, 1, 1, 0),
        # the benchmark's batch and context with all heads of a layer on this device
        _latent("latent 32x8192 128h", 32, 128, 512, 64, 8192, 8192, 1, 1, 0),
        # the same with the heads shared out over eight devices
        _latent("latent 32x8192 16h", 32, 16, 512, 64, 8192, 8192, 1, 1, 0),
        # a continuous batch with small trees of drafted tokens
        _latent("latent ragged 64 64h n1-4", 64, 64, 512, 64, 16, 16384, 1, 4, 2),
        # long contexts at a small batch, one drafted token
        _latent("latent 4x131072 32h n2", 4, 32, 512, 64, 131072, 131072, 2, 2, 1),
        # a smaller model: a narrower latent vector and rotary key
        _latent("latent 8x4096 40h 256+32", 8, 40, 256, 32, 4096, 4096, 1, 1, 0),
        # chains of three drafted tokens, all heads: the most rows
        _latent("latent 32x2048 128h n4", 32, 128, 512, 64, 2048, 2048, 4, 4, 1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("rotary", "latent_append", "latent", "latent"))
    if kind == "rotary":
        while True:
            Hkv = rng.choice((1, 2, 4, 5, 8, 16, 32))
            D = rng.choice((64, 128))
            T = _log(rng, 1, 8192)
            c = _rotary(None, T, Hkv * rng.choice((1, 2, 3, 4, 7, 8)), Hkv, D,
                        rng.choice((D, D, D // 2, D // 4)), rng.random() < 0.5,
                        rng.choice((1, 16, 512)), _log(rng, 1000, 1000000),
                        rng.choice((10000.0, 500000.0, 1000000.0)), rng.choice((1.0, 4.0, 32.0)),
                        rng.random() < 0.6, rng.random() < 0.4)
            if T * (c["Hq"] + Hkv) * D <= 8192 * 40 * 128:
                return c
    if kind == "latent_append":
        while True:
            L = rng.choice((256, 512))
            c = _lappend(None, _log(rng, 1, 8192), rng.choice((1, 8, 16, 20, 40, 64, 128)), L,
                         rng.choice((32, 64)), rng.random() < 0.5, rng.random() < 0.7,
                         rng.choice((1, 16, 512)), _log(rng, 1000, 1000000),
                         rng.choice((1.0, 4.0, 40.0)))
            if c["T"] * (L + c["H"] * c["R"]) <= 8192 * (512 + 16 * 64):
                return c
    while True:
        hi = _log(rng, 20, 100000)
        n_hi = rng.choice((1, 1, 2, 3, 4, 8, 16))
        width = rng.choice((0, 1)) if n_hi == 1 else rng.choice((1, 1, 2, 4))
        c = _latent(None, _log(rng, 1, 64), rng.choice((1, 5, 8, 16, 20, 32, 40, 64, 128)),
                    rng.choice((256, 512, 512)), rng.choice((32, 64, 64)),
                    rng.choice((hi, max(1, hi // 20), 1)), hi,
                    1 if width == 0 else rng.choice((1, n_hi)), n_hi, width)
        w = work(c)
        if w["bytes"] < 6.0e8 and w["flops"] < 7.2e10:
            return c


# --------------------------------------------------------------------- inputs

def _frequencies(rot, theta, factor):
    """Radians a position of each pair, and the magnitude of the rotated values: above a factor of
    one the slow pairs are slowed down by it and the fast ones kept (a ramp between)."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = theta ** (-2.0 * i / rot)
    if factor == 1.0:
        return f.astype(np.float32), 1.0
    ramp = np.clip((i / max(1, rot // 2 - 1) - 0.3) / 0.4, 0.0, 1.0)
    return (f * (1.0 - ramp) + f / factor * ramp).astype(np.float32), 0.1 * math.log(factor) + 1.0


def _positions(rng, T, chunk, far):
    """Positions of T tokens, `chunk` consecutive ones of each sequence."""
    n = -(-T // chunk)
    first = rng.integers(0, max(1, far - chunk), size=n)
    return (first[:, None] + np.arange(chunk)).reshape(-1)[:T].astype(np.int64)


def _slots(rng, T, chunk):
    """Slots of T tokens in a pool whose blocks are handed out in random order; a batch of more
    than 8 tokens holds one padding token."""
    n = -(-T // chunk)
    per = -(-chunk // BLOCK)
    NB = n * per + 3
    blocks = rng.permutation(NB)[:n * per].reshape(n, per)
    at = np.arange(chunk)
    off = rng.integers(0, BLOCK, size=(n, 1)) if chunk == 1 else np.zeros((n, 1), dtype=np.int64)
    slots = (blocks[:, at // BLOCK] * BLOCK + at % BLOCK + off).reshape(-1)[:T].astype(np.int64)
    if T > 8:
        slots[T // 2] = -1
    return slots, NB


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return {"rotary": _prepare_rotary, "latent_append": _prepare_lappend,
            "latent": _prepare_latent}[case["op"]](case, rng, gen)


def _prepare_rotary(c, rng, gen):
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    slots, NB = _slots(rng, T, c["chunk"])
    freq, mag = _frequencies(c["rot"], c["theta"], c["factor"])
    if c["packed"]:
        # one projection's output: queries, keys and values of a token side by side
        qkv = _randn((T, Hq + 2 * Hkv, D), gen).to(torch.bfloat16)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (_randn((T, h, D), gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    shape = (NB, Hkv, BLOCK, D)
    scale = 6.0 / 448 if c["fp8"] else 1.0
    kc, vc = (_randn(shape, gen) for _ in range(2))
    if c["fp8"]:
        kc, vc = ((x / scale).clamp_(-448, 448).to(torch.float8_e4m3fn) for x in (kc, vc))
    else:
        kc, vc = kc.to(torch.bfloat16), vc.to(torch.bfloat16)
    s = {"op": "rotary", "case": c, "q": q, "k": k, "v": v, "kc": kc, "vc": vc, "scale": scale,
         "slots": _cuda(slots), "positions": _cuda(_positions(rng, T, c["chunk"], c["far"])),
         "freq": _cuda(freq), "mag": mag,
         "q_out": torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")}
    if own:
        _pk()
    return s


def _prepare_lappend(c, rng, gen):
    T, H, L, R = c["T"], c["H"], c["L"], c["R"]
    slots, NB = _slots(rng, T, c["chunk"])
    freq, mag = _frequencies(R, 10000.0, c["factor"])
    # one projection's output: the latent vector and the key's rotary part side by side; likewise
    # the queries' two parts, of which the rotary one is wanted here
    down = (_randn((T, L + R), gen) * 1.7).to(torch.bfloat16)
    qp = _randn((T, H, 2 * R + R), gen).to(torch.bfloat16)
    s = {"op": "latent_append", "case": c, "latent": down[:, :L], "k_rope": down[:, L:],
         "q_rope": qp[..., 2 * R:],
         "weight": (1.0 + 0.2 * _randn((L,), gen)).to(torch.bfloat16) if c["norm"] else None,
         "cache": _randn((NB, BLOCK, L + R), gen).to(torch.bfloat16), "slots": _cuda(slots),
         "positions": _cuda(_positions(rng, T, c["chunk"], c["far"])), "freq": _cuda(freq),
         "mag": mag,
         # the attention's queries, whose latent part another product fills
         "q": torch.zeros((T, H, L + R), dtype=torch.bfloat16, device="cuda")}
    if own:
        _pk()
    return s


def _tree(rng, n, width):
    """Parents of a random tree in level order: node 0 is the root, every other node's parent
    comes before it, at most `width` children each."""
    parents, kids, first = [-1], [0], 0
    for _ in range(1, n):
        while kids[first] >= width:
            first += 1
        par = int(rng.integers(first, min(first + 3, len(parents))))
        while kids[par] >= width:
            par = first
        parents.append(par)
        kids.append(0)
        kids[par] += 1
    return parents


def _latent_sizes(c):
    """Nodes and context lengths of each sequence: they belong to the case, whatever the seed, so
    that outputs keep their shapes."""
    sizes = np.random.default_rng(c["B"] * 1009 + c["ctx_hi"] * 31 + c["nodes_hi"])
    counts = sizes.integers(c["nodes_lo"], c["nodes_hi"] + 1, size=c["B"])
    if c["ctx_lo"] >= c["ctx_hi"]:
        lens = np.full(c["B"], c["ctx_hi"], dtype=np.int64)
    else:
        lens = np.exp(sizes.uniform(math.log(c["ctx_lo"]), math.log(c["ctx_hi"] + 1), size=c["B"]))
        lens = np.clip(np.floor(lens).astype(np.int64), c["ctx_lo"], c["ctx_hi"])
    return counts, lens + counts


def _prepare_latent(c, rng, gen):
    B, H, W = c["B"], c["H"], c["L"] + c["R"]
    counts, lens = _latent_sizes(c)
    starts = np.zeros(B + 1, dtype=np.int32)
    starts[1:] = np.cumsum(counts)
    total, N = int(starts[-1]), int(counts.max())
    need = -(-lens // BLOCK)
    NB = int(need.sum() * 1.05) + 2
    perm = rng.permutation(NB).astype(np.int32)
    bt = np.full((B, int(need.max())), -1, dtype=np.int32)
    at = 0
    for s, k in enumerate(need):
        bt[s, :k] = perm[at:at + k]
        at += int(k)
    parents = None
    if c["width"] > 1:
        parents = np.asarray([p for n in counts for p in _tree(rng, int(n), c["width"])],
                             dtype=np.int32)
    # scores of a few units: queries in the latent space are longer than those of a head
    q = _randn((total, H, W), gen) * 1.5
    cache = torch.empty((NB, BLOCK, W), dtype=torch.bfloat16, device="cuda")
    for a in range(0, NB, 4096):
        cache[a:a + 4096] = _randn(tuple(cache[a:a + 4096].shape), gen).to(torch.bfloat16)
    s = {"op": "latent", "case": c, "cache": cache, "q": q.to(torch.bfloat16), "bt": _cuda(bt),
         "lens": _cuda(lens.astype(np.int32)), "scale": 2.0 * W ** -0.5,
         "starts": _cuda(starts) if c["width"] > 0 else None,
         "parents": _cuda(parents) if parents is not None else None, "max_nodes": N,
         # by host data that the program has anyway: the node of each row of a padded batch
         "counts": _cuda(counts.astype(np.int64)),
         "node_row": _cuda(np.minimum(starts[:-1, None] + np.arange(N), total - 1)),
         "row_node": _cuda(np.concatenate([i * N + np.arange(n) for i, n in enumerate(counts)])),
         "out": torch.empty((total, H, c["L"]), dtype=torch.bfloat16, device="cuda")}
    if own:
        pk = _pk()
        s["ws"] = pk.alloc_latent_workspace(B, N, H, c["L"], c["R"])
    return s


# ------------------------------------------------------------------------ run

def run(state):
    return {"rotary": _run_rotary, "latent_append": _run_lappend, "latent": _run_latent}[
        state["op"]](state)


def _rotate(x, positions, freq, mag, inter, rot):
    """The first `rot` elements of each vector of x [T, heads, D], in pairs, turned by the angle
    position * freq and scaled by `mag`; the others as they are.  32 bits, angles in 64."""
    angle = positions.double()[:, None] * freq.double()[None]
    cos = (torch.cos(angle) * mag).float()[:, None]
    sin = (torch.sin(angle) * mag).float()[:, None]
    x = x.float()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _run_rotary(s):
    c = s["case"]
    if own:
        _pk().kv_append_rotary(s["q_out"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"],
                               s["positions"], s["freq"], interleaved=c["inter"],
                               magnitude=s["mag"], k_scale=s["scale"], v_scale=s["scale"])
        return s["q_out"], s["kc"], s["vc"]
    args = (s["positions"], s["freq"], s["mag"], c["inter"], c["rot"])
    s["q_out"].copy_(_rotate(s["q"], *args))
    live = s["slots"] >= 0
    blk, off = s["slots"][live] // BLOCK, s["slots"][live] % BLOCK
    for cache, x in ((s["kc"], _rotate(s["k"], *args)), (s["vc"], s["v"].float())):
        x = x[live]
        if c["fp8"]:
            codes = (x / s["scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[blk, :, off] = codes.view(torch.uint8)
        else:
            cache[blk, :, off] = x.to(torch.bfloat16)
    return s["q_out"], s["kc"], s["vc"]


def _run_lappend(s):
    c = s["case"]
    L = c["L"]
    if own:
        _pk().kv_latent_append(s["q"][..., L:], s["q_rope"], s["latent"], s["k_rope"], s["cache"],
                               s["slots"], s["positions"], s["freq"], norm_weight=s["weight"],
                               eps=EPS, interleaved=c["inter"], magnitude=s["mag"])
        return s["q"], s["cache"]
    args = (s["positions"], s["freq"], s["mag"], c["inter"], c["R"])
    s["q"][..., L:] = _rotate(s["q_rope"], *args).to(torch.bfloat16)
    x = s["latent"].float()
    if s["weight"] is not None:
        x = x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    row = torch.cat((x, _rotate(s["k_rope"][:, None], *args)[:, 0]), dim=1)
    live = s["slots"] >= 0
    s["cache"][s["slots"][live] // BLOCK, s["slots"][live] % BLOCK] = row[live].to(torch.bfloat16)
    return s["q"], s["cache"]


def _run_latent(s):
    if own:
        _pk().paged_latent_attention(s["out"], s["q"], s["cache"], s["bt"], s["lens"], s["scale"],
                                     s["ws"], node_starts=s["starts"], parents=s["parents"],
                                     max_nodes=s["max_nodes"])
        return s["out"]
    c = s["case"]
    B, H, L, N = c["B"], c["H"], c["L"], s["max_nodes"]
    bt = s["bt"].clamp(min=0).long()
    Lp = bt.shape[1] * BLOCK
    kv = s["cache"][bt].float().reshape(B, Lp, -1)                  # [B, Lp, W]
    q = s["q"][s["node_row"]].float().reshape(B, N * H, -1)
    lens, dev = s["lens"].long(), kv.device
    anc = torch.zeros((B, N, N), device=dev)
    if s["parents"] is None:
        anc += torch.tril(torch.ones((N, N), device=dev))
    else:
        # ancestors of each node (itself among them), by doubling along the parents
        par = s["parents"][s["node_row"]].long()
        up = torch.where(par >= 0, par, torch.arange(N, device=dev)[None])
        anc.scatter_(2, up[..., None], 1.0)
        anc = torch.maximum(anc, torch.eye(N, device=dev)[None])
        for _ in range(max(1, N.bit_length())):
            anc = (anc @ anc).clamp(max=1.0)
    pos = torch.arange(Lp, device=dev)
    node = pos[None] - (lens - s["counts"])[:, None]                # [B, Lp]
    seen = torch.gather(anc, 2, node.clamp(0, N - 1)[:, None].expand(B, N, Lp)) > 0
    seen = (node < 0)[:, None] | (seen & ((node >= 0) & (pos[None] < lens[:, None]))[:, None])
    x = (q @ kv.transpose(1, 2)).mul_(s["scale"]).reshape(B, N, H, Lp)
    x.masked_fill_(~seen[:, :, None], -math.inf)
    x = torch.exp_(x.sub_(x.amax(dim=-1, keepdim=True)))
    o = (x.reshape(B, N * H, Lp) @ kv[..., :L]) / x.sum(dim=-1).reshape(B, N * H, 1)
    return o.reshape(B * N, H, L)[s["row_node"]].to(torch.bfloat16)


# ----------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "rotary":
        T, q, kv = c["T"], c["T"] * c["Hq"] * c["D"], c["T"] * c["Hkv"] * c["D"]
        return {"bytes": 4 * q + 2 * kv * (3 if c["fp8"] else 4) + 16 * T,
                "flops": 3.0 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "latent_append":
        T, L, R = c["T"], c["L"], c["R"]
        return {"bytes": 4 * T * (L + R) + 4 * T * c["H"] * R + 16 * T + 2 * L,
                "flops": 4.0 * T * L + 3.0 * T * (c["H"] + 1) * R}
    counts, lens = _latent_sizes(c)
    L, R, H = c["L"], c["R"], c["H"]
    return {"bytes": 2.0 * int(lens.sum()) * (L + R) + 2.0 * int(counts.sum()) * H * (2 * L + R),
            "flops": 2.0 * int((counts * lens).sum()) * H * (2 * L + R)}


# ---------------------------------------------------------------------- exact

def _turn64(x, positions, freq, mag, inter):
    """Pairs as complex numbers, times mag * e^(i angle)."""
    n = freq.numel()
    x = x.double().clone()
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n),
                                                                           slice(n, 2 * n))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous())
    angle = positions.double()[:, None, None] * freq.double()
    z = z * torch.polar(torch.full_like(angle, mag), angle)
    x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rotary":
        turn = (s["positions"], s["freq"], s["mag"], c["inter"])
        out = [_turn64(s["q"], *turn)]
        for cache, x in ((s["kc"], _turn64(s["k"], *turn)), (s["vc"], s["v"].double())):
            held = cache.float().double().transpose(1, 2).flatten(0, 1)      # [slots, Hkv, D]
            for t0 in range(0, c["T"], 1024):
                at = s["slots"][t0:t0 + 1024]
                keep = at >= 0
                held[at[keep]] = (x[t0:t0 + 1024][keep] / s["scale"]).clamp(
                    -448 if c["fp8"] else -math.inf, 448 if c["fp8"] else math.inf)
            out.append(held.unflatten(0, (-1, BLOCK)).transpose(1, 2).contiguous())
        return tuple(out)
    if c["op"] == "latent_append":
        turn = (s["positions"], s["freq"], s["mag"], c["inter"])
        q, held = s["q"].double(), s["cache"].double().flatten(0, 1)
        q[..., c["L"]:] = _turn64(s["q_rope"], *turn)
        x = s["latent"].double()
        if c["norm"]:
            x = x / (x.square().sum(dim=1, keepdim=True) / c["L"] + EPS).sqrt()
            x = x * s["weight"].double()
        k = _turn64(s["k_rope"][:, None], *turn)[:, 0]
        keep = s["slots"] >= 0
        held[s["slots"][keep], :c["L"]] = x[keep]
        held[s["slots"][keep], c["L"]:] = k[keep]
        return q, held.unflatten(0, (-1, BLOCK))
    # attention: one sequence after the other, the tree's mask from a walk along the parents
    counts, lens = _latent_sizes(c)
    H, L = c["H"], c["L"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    parents = None if s["parents"] is None else s["parents"].cpu().numpy()
    t0 = 0
    for b in range(c["B"]):
        n, ctx = int(counts[b]), int(lens[b])
        mask = torch.zeros((n, ctx), dtype=torch.float64)
        mask[:, ctx - n:] = -math.inf
        for i in range(n):
            j = i
            while j >= 0:
                mask[i, ctx - n + j] = 0.0
                j = j - 1 if parents is None else int(parents[t0 + j])
        mask = mask.cuda()
        kv = s["cache"][s["bt"][b, :-(-ctx // BLOCK)].long()].double().flatten(0, 1)[:ctx]
        for i in range(n):
            x = s["q"][t0 + i].double() @ kv.t() * s["scale"] + mask[i]
            out[t0 + i] = torch.softmax(x, dim=1) @ kv[:, :L]
        t0 += n
    return out
