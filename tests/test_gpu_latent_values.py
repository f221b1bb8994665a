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
