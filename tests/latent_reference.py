"""Plain 64-bit implementations of rotary positions, the latent append and attention over a
latent cache, for the tests, with bounds on what the library's roundings may cost.  Nothing here
shares code with the library."""
import numpy as np
import torch

from tree_reference import ancestors

BS = 16
HALF_BF16 = 2.0 ** -8           # half a step of bfloat16, relative to the value


def turn(x, positions, freq, mag, interleaved):
    """x [T, heads, D] float64, the first 2 * len(freq) elements turned: (values, sums of the
    pair's absolute values, zero behind the pairs)."""
    x = x.double()
    n = len(freq)
    i = torch.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    t = positions.double()[:, None, None] * freq.double()
    y, size = x.clone(), torch.zeros_like(x)
    y[..., a] = mag * (x[..., a] * torch.cos(t) - x[..., b] * torch.sin(t))
    y[..., b] = mag * (x[..., b] * torch.cos(t) + x[..., a] * torch.sin(t))
    size[..., a] = size[..., b] = mag * (x[..., a].abs() + x[..., b].abs())
    return y, size


def turn_error(size):
    """What float32 may cost before the rounding of the result.  An angle is a 32-bit fraction of
    a turn rounded to float32 (2^-24 of at most pi: 2^-22.3), its sine and cosine are off by an
    ulp (2^-23), the magnitude's product, the two products and the sum by 2^-24 each: less than
    2^-20.9 of the pair's absolute values."""
    return size * 2.0 ** -20


def norm(x, weight, eps):
    x = x.double()
    if weight is None:
        return x
    return x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + eps) * weight.double()


def attention(q, cache, bt, lens, starts, parents, scale, L):
    """q [T, H, W], cache [NB, 16, W] (bfloat16) -> (out [T, H, L], bound), float64.

    The bound counts: weights rounded to bfloat16, 2^-8 each, their sum that of the rounded ones,
    so that the result moves by 2^-8 (sum w |v| + |o|) at most; the score's 36 or fewer partial
    sums and the product's, one for 16 keys, each off by 2^-23 of what they add up in absolute
    value (a score's error is a weight's relative error, twice with the sum's); exponentials,
    references and factors of joined parts by 2^-20 in all; the output by 2^-8."""
    T, H, W = q.shape
    out = torch.zeros((T, H, L), dtype=torch.float64)
    bound = torch.zeros_like(out)
    q, cache = q.double(), cache.double()
    for s in range(len(lens)):
        t0, n, ctx = int(starts[s]), int(starts[s + 1] - starts[s]), int(lens[s])
        if n == 0 or ctx == 0:
            continue
        c = cache[torch.as_tensor(bt[s, :-(-ctx // BS)]).long()].flatten(0, 1)[:ctx]
        par = (np.arange(n) - 1 if parents is None else np.asarray(parents[t0:t0 + n])).astype(int)
        base = ctx - n
        for i, seen in enumerate(ancestors(par)):
            if par[i] == -2:
                continue
            idx = torch.cat([torch.arange(base), base + torch.tensor(sorted(seen))]).long()
            rows = c[idx]
            x = q[t0 + i] @ rows.T * scale
            w = torch.softmax(x, dim=1)
            o = w @ rows[:, :L]
            size = w @ rows[:, :L].abs()
            off = (abs(scale) * (q[t0 + i].abs() @ rows.abs().T)).amax(dim=1, keepdim=True)
            rel = 2 * 36 * 2.0 ** -23 * off + (len(idx) / 16 + 1) * 2.0 ** -23 + 2.0 ** -20
            out[t0 + i] = o
            bound[t0 + i] = 2 * HALF_BF16 * o.abs() + (HALF_BF16 + rel) * size
    return out, bound * 1.01
