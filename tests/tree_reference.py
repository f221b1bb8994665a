"""Plain 64-bit implementations of the draft-tree operations, for the tests:
attention by the formula, verification by the sequential rule, compaction by
copying.  Nothing here shares code with the library."""
import numpy as np

BS = 16


def e4m3_values():
    """The value of each of the 256 E4M3 codes (bias 7, no infinities)."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = np.nan if (e == 15 and m == 7) else (m / 8 * 2.0 ** -6 if e == 0
                                                 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -x if s else x
    return v


def random_tree(rng, n, width=3, pads=0.0):
    """Parents of a random tree of n nodes in topological order; with pads > 0
    some nodes (never the first) are padding."""
    par = np.full(n, -1, dtype=np.int32)
    for i in range(1, n):
        par[i] = i - 1 if width == 1 else rng.integers(max(0, i - 2 * width), i)
        if rng.random() < pads:
            par[i] = -2
    return par


def ancestors(par):
    """seen[i] = the nodes node i sees within its tree (itself among them)."""
    seen = []
    for i in range(len(par)):
        mine, a = set(), i
        while a >= 0 and par[a] != -2:
            mine.add(a)
            a = int(par[a])
        seen.append(set() if par[i] == -2 else mine)
    return seen


def attention(q, k, v, bt, lens, starts, parents, scale):
    """q [T, Hq, D], k / v [NB, Hkv, 16, D], all float64 -> [T, Hq, D]."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out = np.zeros((T, Hq, D))
    for s in range(len(lens)):
        t0, n, L = int(starts[s]), int(starts[s + 1] - starts[s]), int(lens[s])
        if n == 0 or L == 0:
            continue
        pages = bt[s, :-(-L // BS)]
        ks = k[pages].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L]
        vs = v[pages].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L]
        par = (np.arange(n) - 1 if parents is None else parents[t0:t0 + n]).astype(int)
        base = L - n
        for i, seen in enumerate(ancestors(par)):
            if par[i] == -2:
                continue
            idx = np.concatenate([np.arange(base), base + np.array(sorted(seen), dtype=int)])
            for h in range(Hkv):
                x = q[t0 + i, h * G:(h + 1) * G] @ ks[h, idx].T * scale
                x = np.exp(x - x.max(axis=1, keepdims=True))
                out[t0 + i, h * G:(h + 1) * G] = (x @ vs[h, idx]) / x.sum(axis=1, keepdims=True)
    return out


def verify(target, draft, tokens, parents, starts, accept_u, sample_u, max_nodes, greedy=False):
    """The walk of kv_tree_verify, one sequence after the other, in float64:
    (accept_lens, accept_nodes, out_tokens)."""
    B, V = len(starts) - 1, target.shape[1]
    lens = np.zeros(B, dtype=np.int32)
    nodes = np.full((B, max_nodes), -1, dtype=np.int32)
    toks = np.full((B, max_nodes), -1, dtype=np.int32)

    def clean(x):
        x = x.astype(np.float64)
        return np.where((x > 0) & (x < np.inf), x, 0.0)

    for s in range(B):
        t0, n = int(starts[s]), int(starts[s + 1] - starts[s])
        if n == 0:
            continue
        par = (np.arange(n) - 1 if parents is None else parents[t0:t0 + n]).astype(int)
        path, v = [0], 0
        while True:
            kids = [c for c in range(v + 1, n) if par[c] == v]
            took = None
            if greedy:
                row = target[t0 + v].astype(np.float64)
                row = np.where(np.isnan(row), -np.inf, row)
                last = int(np.argmax(row))
                for c in kids:
                    if tokens[t0 + c] == last:
                        took = c
                        break
            else:
                p = clean(target[t0 + v])
                q = None if draft is None else clean(draft[t0 + v])
                R, Z, a = p.copy(), 1.0, 0.0
                for c in kids:
                    x = int(tokens[t0 + c])
                    if not 0 <= x < V:
                        continue
                    qx = 1.0 if q is None else q[x]
                    if float(accept_u[t0 + c]) * qx * Z < R[x]:
                        took = c
                        break
                    if q is None:
                        Z -= R[x]
                        R[x] = 0.0
                    else:
                        a += Z
                        R = np.maximum(p - a * q, 0.0)
                        Z = R.sum()
                if took is None:
                    if R.sum() <= 0:
                        R = p
                    cum = np.cumsum(R)
                    above = np.nonzero(cum > float(sample_u[s]) * cum[-1])[0]
                    pos = np.nonzero(R > 0)[0]
                    last = -1 if len(pos) == 0 else int(above[0] if len(above) else pos[-1])
            if took is None:
                break
            path.append(took)
            v = took
        lens[s] = len(path)
        nodes[s, :len(path)] = path
        toks[s, :len(path)] = [int(tokens[t0 + c]) for c in path[1:]] + [last]
    return lens, nodes, toks


def compact(k, v, bt, lens, starts, nodes, accept):
    """Caches after the accepted nodes' vectors have moved (copies)."""
    k, v = k.copy(), v.copy()
    for s in range(len(lens)):
        n = int(starts[s + 1] - starts[s])
        base = int(lens[s]) - n
        for c in (k, v):
            old = c.copy()
            for i in range(int(accept[s])):
                sp, dp = base + int(nodes[s, i]), base + i
                c[bt[s, dp // BS], :, dp % BS] = old[bt[s, sp // BS], :, sp % BS]
    return k, v
