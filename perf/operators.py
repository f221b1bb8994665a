"""Cases, plain forms and exact values of the draft-tree operators: attention of a tree of drafted
tokens over the paged cache, verification of the tree against the target's probabilities, and
compaction of the accepted tokens' K/V.  ``run`` is the plain form while ``own`` is false and the
library's call while it is true."""
import math

import numpy as np
import torch

own = False

BLOCK = 16


def _pk():
    import paged_kv_cache_21_gb300 as pk
    return pk


# ---------------------------------------------------------------------- cases

def _attend(name, B, Hq, Hkv, D, ctx_lo, ctx_hi, nodes_lo, nodes_hi, width, fp8=False):
    c = {"op": "attend", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
         "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "width": width, "fp8": fp8}
    if name:
        c["name"] = name
    return c


def _verify(name, B, V, nodes, width, draft, greedy, bf16=False):
    c = {"op": "verify", "B": B, "V": V, "nodes": nodes, "width": width, "draft": draft,
         "greedy": greedy, "bf16": bf16}
    if name:
        c["name"] = name
    return c


def _compact(name, layers, B, Hkv, D, ctx, nodes, accept, fp8=False):
    c = {"op": "compact", "layers": layers, "B": B, "Hkv": Hkv, "D": D, "ctx": ctx,
         "nodes": nodes, "accept": accept, "fp8": fp8}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one request on a tiny model: the latency of the call
        _attend("attend 1x128 4q/1kv d64 n5", 1, 4, 1, 64, 128, 128, 5, 5, 1),
        # the benchmark's layer (32 x 8192, 32q/8kv) with a small tree per request
        _attend("attend 32x8192 32q/8kv n8", 32, 32, 8, 128, 8192, 8192, 8, 8, 3),
        # the same layer with an E4M3 cache
        _attend("attend 32x8192 e4m3 n16", 32, 32, 8, 128, 8192, 8192, 16, 16, 4, fp8=True),
        # a continuous batch: lengths log-uniform, trees of 1 to 32 nodes
        _attend("attend ragged 64 32q/8kv n1-32", 64, 32, 8, 128, 16, 16384, 1, 32, 4),
        # long contexts at a small batch (64q/8kv)
        _attend("attend 4x131072 64q/8kv n4", 4, 64, 8, 128, 131072, 131072, 4, 4, 2),
        # full multi-head attention: one query head per KV head
        _attend("attend 8x4096 32q/32kv n12", 8, 32, 32, 128, 4096, 4096, 12, 12, 3),
        # the benchmark's layer with a wide tree: the most arithmetic
        _attend("attend 32x8192 32q/8kv n64", 32, 32, 8, 128, 8192, 8192, 64, 64, 8),
        # one request, a drafted chain, a small vocabulary: the latency of the call
        _verify("verify 1 chain n5 V32000", 1, 32000, 5, 1, True, False),
        # a batch of trees with the draft model's distributions
        _verify("verify 64 trees n26 V128000", 64, 128000, 26, 4, True, False),
        # greedy decoding: the target's largest entry along the path
        _verify("verify 32 greedy n16 V100003", 32, 100003, 16, 3, False, True),
        # one request, all layers of a model
        _compact("compact 1 x 32 layers", 32, 1, 8, 128, 300, 8, 4),
        # a large batch, all layers of a model
        _compact("compact 64 x 32 layers", 32, 64, 8, 128, 250, 48, 7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("attend", "attend", "verify", "compact"))
    if kind == "attend":
        while True:
            Hkv = rng.choice((1, 2, 4, 5, 8, 16, 32))
            G = rng.choice((1, 2, 3, 4, 7, 8, 16))
            hi = _log(rng, 20, 60000)
            n_hi = _log(rng, 1, 64)
            c = _attend(None, _log(rng, 1, 64), Hkv * G, Hkv, rng.choice((64, 128)),
                        rng.choice((hi, max(1, hi // 20), 1)), hi, rng.choice((1, n_hi)), n_hi,
                        rng.choice((1, 2, 4, 8)), rng.random() < 0.4)
            if Hkv * G <= 128 and _attend_bytes(c) < 2.0e9 and _attend_flops(c) < 2.5e11:
                return c
    if kind == "verify":
        nodes = _log(rng, 1, 64)
        while True:
            c = _verify(None, _log(rng, 1, 64), _log(rng, 500, 160000), nodes,
                        rng.choice((1, 2, 4, 6)), rng.random() < 0.6, rng.random() < 0.25,
                        rng.random() < 0.3)
            if c["B"] * c["V"] * nodes < 2.0e8:
                return c
    while True:
        nodes = _log(rng, 2, 64)
        c = _compact(None, _log(rng, 1, 64), _log(rng, 1, 64), rng.choice((1, 2, 4, 8, 16)),
                     rng.choice((64, 128)), rng.randint(0, 300), nodes,
                     rng.randint(1, max(1, nodes // 3)), rng.random() < 0.4)
        tokens = c["layers"] * c["B"] * (c["ctx"] + nodes + BLOCK)
        if tokens * c["Hkv"] * c["D"] < 3.5e8:
            return c


# --------------------------------------------------------------------- inputs

def _tree(rng, n, width):
    """Parents of a random tree in level order: node 0 is the root, every other node's parent
    comes before it, at most `width` children each (width 1: a chain)."""
    parents = [-1]
    kids = [0]
    first = 0
    for _ in range(1, n):
        if width == 1:
            par = len(parents) - 1
        else:
            while kids[first] >= width:
                first += 1
            par = int(rng.integers(first, min(first + 3, len(parents))))
            while kids[par] >= width:
                par = first
        parents.append(par)
        kids.append(0)
        kids[par] += 1
    return parents


def _trees(rng, counts, width):
    starts = np.zeros(len(counts) + 1, dtype=np.int32)
    starts[1:] = np.cumsum(counts)
    parents = [p for n in counts for p in _tree(rng, int(n), width)]
    return starts, np.asarray(parents, dtype=np.int32)


def _lengths(rng, lo, hi, B):
    if lo >= hi:
        return np.full(B, hi, dtype=np.int64)
    x = np.floor(np.exp(rng.uniform(math.log(lo), math.log(hi + 1), size=B))).astype(np.int64)
    return np.clip(x, lo, hi)


def _pages(rng, lens):
    """Block tables of a pool whose pages are handed out in random order."""
    need = -(-lens // BLOCK)
    NB = int(need.sum() * 1.05) + 2
    perm = rng.permutation(NB).astype(np.int32)
    bt = np.full((len(lens), int(need.max())), -1, dtype=np.int32)
    at = 0
    for s, k in enumerate(need):
        bt[s, :k] = perm[at:at + k]
        at += int(k)
    return bt, NB


def _normal(shape, gen, fp8):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x.to(torch.float8_e4m3fn) if fp8 else x.to(torch.bfloat16)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return {"attend": _prepare_attend, "verify": _prepare_verify,
            "compact": _prepare_compact}[case["op"]](case, rng, gen)


def _attend_sizes(c):
    """Nodes and context lengths of each sequence: they belong to the case, whatever the seed, so
    that outputs keep their shapes."""
    sizes = np.random.default_rng(c["B"] * 1009 + c["ctx_hi"] * 31 + c["nodes_hi"])
    counts = sizes.integers(c["nodes_lo"], c["nodes_hi"] + 1, size=c["B"])
    return counts, _lengths(sizes, c["ctx_lo"], c["ctx_hi"], c["B"]) + counts


def _compact_sizes(c):
    """Context lengths, accepted nodes of each sequence and how many of them lie in their place."""
    B, n, m = c["B"], c["nodes"], min(c["accept"], c["nodes"])
    sizes = np.random.default_rng(B * 1009 + c["ctx"] * 31 + n)
    lens = np.maximum(0, c["ctx"] - sizes.integers(0, 40, size=B)) + n
    k = sizes.integers(max(1, m // 2), m + 1, size=B)
    here = np.maximum(sizes.integers(1, k + 1), k - (n - k))
    return lens, k, here


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _prepare_attend(c, rng, gen):
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    counts, lens = _attend_sizes(c)
    starts, parents = _trees(rng, counts, c["width"])
    bt, NB = _pages(rng, lens)
    total = int(starts[-1])
    # the scales of an E4M3 cache of normal values: amax / 448
    ks = vs = 4.25 / 448 if c["fp8"] else 1.0
    shape = (NB, Hkv, BLOCK, D)
    kc, vc = ((_normal(shape, gen, False).float() / ks).clamp_(-448, 448).to(torch.float8_e4m3fn)
              if c["fp8"] else _normal(shape, gen, False) for _ in range(2))
    s = {"op": "attend", "case": c, "kc": kc, "vc": vc, "ks": ks, "vs": vs,
         "q": _normal((total, Hq, D), gen, False), "bt": _cuda(bt),
         "lens": _cuda(lens.astype(np.int32)), "starts": _cuda(starts), "parents": _cuda(parents),
         "max_nodes": int(counts.max()), "scale": D ** -0.5,
         # by host data that the program has anyway: the node of each row of a padded batch
         "node_row": _cuda(np.minimum(starts[:-1, None] + np.arange(counts.max()), total - 1)),
         "row_node": _cuda(np.concatenate([s * counts.max() + np.arange(n)
                                           for s, n in enumerate(counts)])),
         "out": torch.empty((total, Hq, D), dtype=torch.bfloat16, device="cuda")}
    if own:
        pk = _pk()
        s["ws"] = pk.alloc_tree_workspace(B, s["max_nodes"], Hq, Hkv, D,
                                          pk.FP8_E4M3 if c["fp8"] else pk.BF16)
    return s


def _prepare_verify(c, rng, gen):
    B, V, n = c["B"], c["V"], c["nodes"]
    starts, parents = _trees(rng, [n] * B, c["width"])
    total = B * n
    dt = torch.bfloat16 if c["bf16"] else torch.float32
    # a peaked distribution, and a draft model that nearly has it
    logits = torch.randn((total, V), generator=gen, device="cuda") * 2.5
    target = torch.softmax(logits, dim=1).to(dt)
    logits.add_(torch.randn((total, V), generator=gen, device="cuda") * 0.7)
    draft = torch.softmax(logits, dim=1).to(dt)
    # a node's token is drawn from the draft's distribution at its parent (greedy: most often
    # the target's largest entry there)
    par = _cuda(np.maximum(parents, 0) + np.repeat(starts[:-1], n)).long()
    if c["greedy"]:
        tokens = torch.topk(logits, min(8, V), dim=1).indices[par]
        kth = torch.from_numpy(rng.integers(0, min(8, V), size=(total, 1)) // 2).cuda()
        tokens = tokens.gather(1, kth)[:, 0]
    else:
        tokens = torch.multinomial(draft.float()[par], 1, generator=gen)[:, 0]
    del logits
    u = torch.rand((total + B,), generator=gen, device="cuda")
    depth = np.zeros(total, dtype=np.int64)
    kids = np.zeros(total, dtype=np.int64)
    for i in range(total):
        if parents[i] >= 0:
            p = parents[i] + i // n * n
            depth[i] = depth[p] + 1
            kids[p] += 1
    s = {"op": "verify", "case": c, "target": target,
         "draft": draft if c["draft"] and not c["greedy"] else None,
         "tokens": tokens.to(torch.int32), "parents": _cuda(parents), "starts": _cuda(starts),
         "accept_u": u[:total].clone(), "sample_u": u[total:].clone(), "greedy": c["greedy"],
         "depth": int(depth.max()), "kids": int(kids.max()),
         "accept_lens": torch.empty(B, dtype=torch.int32, device="cuda"),
         "accept_nodes": torch.empty((B, n), dtype=torch.int32, device="cuda"),
         "out_tokens": torch.empty((B, n), dtype=torch.int32, device="cuda")}
    if own:
        _pk()
    return s


def _prepare_compact(c, rng, gen):
    B, n = c["B"], c["nodes"]
    lens, accepted, in_place = _compact_sizes(c)
    bt, NB = _pages(rng, lens)
    shape = (c["layers"], NB, c["Hkv"], BLOCK, c["D"])
    kc, vc = _normal(shape, gen, c["fp8"]), _normal(shape, gen, c["fp8"])
    # an accepted path: its first nodes lie where they belong, the others further on in the tree
    # (no source is written, so a repeated pass gives the same caches)
    nodes = np.full((B, n), -1, dtype=np.int32)
    for s in range(B):
        k, here = int(accepted[s]), int(in_place[s])
        nodes[s, :here] = np.arange(here)
        nodes[s, here:k] = np.sort(rng.choice(np.arange(k, n), size=k - here, replace=False))
    s = {"op": "compact", "case": c, "kc": kc, "vc": vc, "bt": _cuda(bt),
         "lens": _cuda(lens.astype(np.int32)),
         "starts": _cuda(np.arange(B + 1, dtype=np.int32) * n), "accept_nodes": _cuda(nodes),
         "accept_lens": _cuda(accepted.astype(np.int32))}
    if own:
        pk = _pk()
        s["layers"] = pk.CacheLayers(list(kc.unbind(0)), list(vc.unbind(0)))
    return s


# ------------------------------------------------------------------------ run

def run(state):
    return {"attend": _run_attend, "verify": _run_verify, "compact": _run_compact}[state["op"]](
        state)


def _run_attend(s):
    if own:
        _pk().paged_tree_attention(s["out"], s["q"], s["kc"], s["vc"], s["bt"], s["lens"],
                                   s["starts"], s["parents"], s["max_nodes"], s["scale"], s["ws"],
                                   s["ks"], s["vs"])
        return s["out"]
    c = s["case"]
    B, Hq, Hkv, D, N = c["B"], c["Hq"], c["Hkv"], c["D"], s["max_nodes"]
    G = Hq // Hkv
    bt = s["bt"].clamp(min=0).long()
    Lp = bt.shape[1] * BLOCK
    # [B, Hkv, Lp, D] in 32 bits
    k = s["kc"][bt].float().transpose(1, 2).reshape(B, Hkv, Lp, D)
    v = s["vc"][bt].float().transpose(1, 2).reshape(B, Hkv, Lp, D)
    q = s["q"][s["node_row"]].float()                               # [B, N, Hq, D]
    q = q.reshape(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    lens = s["lens"].long()
    counts = (s["starts"][1:] - s["starts"][:-1]).long()
    # ancestors of each node (itself among them), by doubling along the parents
    par = s["parents"][s["node_row"]].long()                        # [B, N]
    up = torch.where(par >= 0, par, torch.arange(N, device=par.device)[None])
    anc = torch.zeros((B, N, N), device=par.device)
    anc.scatter_(2, up[..., None], 1.0)
    anc = torch.maximum(anc, torch.eye(N, device=par.device)[None])
    for _ in range(max(1, N.bit_length())):
        anc = (anc @ anc).clamp(max=1.0)
    pos = torch.arange(Lp, device=par.device)
    base = lens - counts
    node = pos[None] - base[:, None]                                # [B, Lp]
    seen = torch.gather(anc, 2, node.clamp(0, N - 1)[:, None].expand(B, N, Lp)) > 0
    seen = (node < 0)[:, None] | (seen & (node >= 0)[:, None] & (pos[None] < lens[:, None])[:, None])
    x = (q @ k.transpose(2, 3)).mul_(s["scale"] * s["ks"]).reshape(B, Hkv, N, G, Lp)
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    x = torch.exp_(x.sub_(x.amax(dim=-1, keepdim=True)))
    o = (x.reshape(B, Hkv, N * G, Lp) @ v) / x.sum(dim=-1).reshape(B, Hkv, N * G, 1) * s["vs"]
    o = o.reshape(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B * N, Hq, D)
    return o[s["row_node"]].to(torch.bfloat16)


def _run_verify(s):
    if own:
        _pk().kv_tree_verify(s["accept_lens"], s["accept_nodes"], s["out_tokens"], s["target"],
                             s["tokens"], s["parents"], s["starts"], s["accept_u"], s["sample_u"],
                             draft_probs=s["draft"], greedy=s["greedy"])
        return s["accept_lens"], s["accept_nodes"], s["out_tokens"]
    c = s["case"]
    B, V, n = c["B"], c["V"], c["nodes"]
    dev = s["tokens"].device
    rows = torch.arange(B, device=dev)
    par, tok = s["parents"].reshape(B, n).long(), s["tokens"].reshape(B, n).long()
    u = s["accept_u"].reshape(B, n).double()
    nodes = torch.full((B, n + 1), -1, dtype=torch.long, device=dev)
    toks = torch.full((B, n + 1), -1, dtype=torch.long, device=dev)
    nodes[:, 0] = 0
    length = torch.ones(B, dtype=torch.long, device=dev)
    v = torch.zeros(B, dtype=torch.long, device=dev)
    done = torch.zeros(B, dtype=torch.bool, device=dev)
    final = torch.zeros(B, dtype=torch.long, device=dev)
    # one level of the tree after the other, the sequences together; a sequence that has stopped
    # keeps what it has
    for _ in range(s["depth"] + 1):
        at = rows * n + v
        p = s["target"][at].double()
        qd = None if s["draft"] is None else s["draft"][at].double()
        kids = par == v[:, None]
        order = torch.cumsum(kids, dim=1)
        best = p.argmax(dim=1)
        a = torch.zeros(B, dtype=torch.double, device=dev)
        Z = torch.ones(B, dtype=torch.double, device=dev)
        R = p.clone()
        took = torch.full((B,), -1, dtype=torch.long, device=dev)
        for k in range(1, s["kids"] + 1):
            is_kid = kids & (order == k)
            live = is_kid.any(dim=1) & (took < 0)
            child = is_kid.long().argmax(dim=1)
            x = tok[rows, child]
            uc = u[rows, child]
            if s["greedy"]:
                ok = live & (x == best)
            else:
                qx = torch.ones_like(uc) if qd is None else qd[rows, x]
                ok = live & (uc * qx * Z < R[rows, x])
                lost = live & ~ok
                if qd is None:
                    Z = torch.where(lost, Z - R[rows, x], Z)
                    R[rows, x] = torch.where(lost, torch.zeros_like(Z), R[rows, x])
                else:
                    a = torch.where(lost, a + Z, a)
                    R = torch.where(lost[:, None], (p - a[:, None] * qd).clamp(min=0), R)
                    Z = torch.where(lost, R.sum(dim=1), Z)
            took = torch.where(ok, child, took)
        if s["greedy"]:
            pick = best
        else:
            R = torch.where(R.sum(dim=1, keepdim=True) > 0, R, p)
            cum = torch.cumsum(R, dim=1)
            pick = (cum <= s["sample_u"].double()[:, None] * cum[:, -1:]).sum(dim=1)
            pick = pick.clamp(max=V - 1)
        go = (took >= 0) & ~done
        toks[rows, torch.where(done, n, length - 1)] = torch.where(
            go, tok[rows, took.clamp(min=0)], pick)
        nodes[rows, torch.where(go, length, n)] = took
        length = length + go
        done = done | ~go
        v = torch.where(go, took, v)
    return length.int(), nodes[:, :n].int(), toks[:, :n].int()


def _run_compact(s):
    if own:
        _pk().kv_tree_compact(s["layers"], s["bt"], s["lens"], s["starts"], s["accept_nodes"],
                              s["accept_lens"])
        return s["kc"], s["vc"]
    base = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1]).long()
    nodes = s["accept_nodes"].long()
    i = torch.arange(nodes.shape[1], device=nodes.device)[None]
    # what is not moved is copied onto itself: every place is written once, and none is left out
    live = i < s["accept_lens"].long()[:, None]
    src = base[:, None] + torch.where(live, nodes, i)
    dst = (base[:, None] + i).expand_as(src)
    bt = s["bt"].long()
    sb, db = torch.gather(bt, 1, src // BLOCK), torch.gather(bt, 1, dst // BLOCK)
    for cache in (s["kc"], s["vc"]):
        w = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
        w[:, db, :, dst % BLOCK] = w[:, sb, :, src % BLOCK]
    return s["kc"], s["vc"]


# ----------------------------------------------------------------------- work

def _attend_bytes(c):
    counts, lens = _attend_sizes(c)
    kv = int(lens.sum()) * c["Hkv"] * c["D"] * 2 * (1 if c["fp8"] else 2)
    return kv + 2 * int(counts.sum()) * c["Hq"] * c["D"] * 2


def _attend_flops(c):
    counts, lens = _attend_sizes(c)
    return 4.0 * int((counts * lens).sum()) * c["Hq"] * c["D"]


def work(case):
    if case["op"] == "attend":
        return {"bytes": _attend_bytes(case), "flops": _attend_flops(case)}
    if case["op"] == "verify":
        # the rows of the node where the walk stops (the others' single entries count for nothing)
        rows = case["B"] * (2 if case["draft"] and not case["greedy"] else 1)
        return {"bytes": rows * case["V"] * (2 if case["bf16"] else 4), "flops": rows * case["V"]}
    # the nodes that move, read and written once in K and V (one at least, for the call itself)
    _, accepted, in_place = _compact_sizes(case)
    moved = max(1, int((accepted - in_place).sum()))
    return {"bytes": 4.0 * case["layers"] * moved * case["Hkv"] * case["D"]
            * (1 if case["fp8"] else 2), "flops": 0}


# ---------------------------------------------------------------------- exact

def exact(case, seed):
    """Attention in 64 bits, one sequence and KV head after the other, the tree's mask from a walk
    along the parents.  The other operators return whole numbers and copies."""
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    Hkv, D, G = case["Hkv"], case["D"], case["Hq"] // case["Hkv"]
    starts, parents = s["starts"].cpu().numpy(), s["parents"].cpu().numpy()
    lens, bt = s["lens"].cpu().numpy(), s["bt"].long()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        t0, n, L = int(starts[b]), int(starts[b + 1] - starts[b]), int(lens[b])
        mask = torch.zeros((n, L), dtype=torch.float64)
        mask[:, L - n:] = -math.inf
        for i in range(n):
            j = i
            while j >= 0:
                mask[i, L - n + j] = 0.0
                j = int(parents[t0 + j])
        mask = mask.cuda().repeat_interleave(G, dim=0)
        pages = bt[b, :-(-L // BLOCK)]
        for h in range(Hkv):
            k = s["kc"][:, h][pages].double().reshape(-1, D)[:L] * s["ks"]
            v = s["vc"][:, h][pages].double().reshape(-1, D)[:L] * s["vs"]
            q = s["q"][t0:t0 + n, h * G:(h + 1) * G].double().reshape(n * G, D)
            w = torch.softmax(q @ k.t() * s["scale"] + mask, dim=1)
            out[t0:t0 + n, h * G:(h + 1) * G] = (w @ v).reshape(n, G, D)
    return out
