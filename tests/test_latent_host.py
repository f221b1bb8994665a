"""Rotary frequencies, sizes of latent caches and what the rotary and latent calls refuse, on the
CPU."""
import ctypes
import math

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build_native()
    import paged_kv_cache_21_gb300 as pk
    return pk


def half_ulp(x):
    return np.abs(x) * 2.0 ** -24


def test_frequencies(pk):
    d, theta = 64, 500000.0
    i = np.arange(d // 2)
    plain = theta ** (-2.0 * i / d)
    f, m = pk.rotary_frequencies(d, theta)
    assert f.dtype == np.float32 and m == 1.0
    # (pow in double twice: 2^-50 beside the rounding to float32)
    def near(got, want):
        assert (np.abs(got - want) <= half_ulp(want) * (1 + 2.0 ** -20)).all()
    near(f, plain)
    near(pk.rotary_frequencies(d, theta, "linear", 8.0)[0], plain / 8)
    near(pk.rotary_frequencies(d, theta, "base", 8.0)[0],
         (theta * 8.0 ** (d / (d - 2))) ** (-2.0 * i / d))
    # the slowest pair of "base" is that of "linear"
    assert abs(pk.rotary_frequencies(d, theta, "base", 8.0)[0][-1] * 8 / plain[-1] - 1) < 1e-6

    f, m = pk.rotary_frequencies(d, theta, "bands", 8.0, 1.0, 4.0, 8192.0)
    turns = 8192 * plain / (2 * math.pi)
    blend = np.clip((turns - 1) / 3, 0, 1)
    near(f, plain * blend + plain / 8 * (1 - blend))
    assert m == 1.0 and (f[turns >= 4] == plain[turns >= 4].astype(np.float32)).all()

    f, m = pk.rotary_frequencies(d, 10000.0, "parts", 16.0, 1.0, 32.0, 4096.0)
    plain = 10000.0 ** (-2.0 * i / d)
    pair = lambda t: d * math.log(4096 / (t * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), d - 1)
    slow = np.clip((i - lo) / (hi - lo), 0, 1)
    near(f, plain * (1 - slow) + plain / 16 * slow)
    assert abs(m - (0.1 * math.log(16.0) + 1)) < 1e-7
    assert (pk.rotary_frequencies(d, 10000.0, "parts", 1.0, 1.0, 32.0, 4096.0)[0]
            == plain.astype(np.float32)).all()


@pytest.mark.parametrize("args", [
    (63,), (0,), (-2,), (64, 0.0), (64, float("nan")), (64, 1e4, "linear", 0.5),
    (64, 1e4, "linear", float("inf")), (2, 1e4, "base", 2.0),
    (64, 1e4, "parts", 2.0, 2.0, 1.0, 4096.0), (64, 1e4, "bands", 2.0, 1.0, 4.0, 0.0),
    (64, 1.0, "parts", 2.0, 1.0, 32.0, 4096.0)])
def test_frequencies_refused(pk, args):
    with pytest.raises(pk.KVError) as e:
        pk.rotary_frequencies(*args)
    assert e.value.code == pk.KV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        pk.rotary_frequencies(64, scaling="other")
    assert pk._lib.kv_rotary_frequencies(None, None, 64, 1e4, 0, 1.0, 1.0, 2.0, 1.0) == \
        pk.KV_ERR_INVALID_ARG


def test_latent_bytes(pk):
    assert pk.latent_bytes(60, 2, 4096, 576) == 60 * 2 * 4096 * 576 * 2
    assert pk.latent_bytes(0, 2, 4096, 576) == 0
    with pytest.raises(ValueError):
        pk.latent_bytes(1, -1, 1, 1)
    with pytest.raises(ValueError):
        pk.latent_bytes(1 << 30, 1 << 30, 1 << 30, 576)


P = ctypes.c_void_p
A = P(4096)


def rotary(pk, q_out=A, so=512, q=A, sq=512, k=A, sk=128, v=A, sv=128, kc=A, vc=A, slots=A, pos=A,
           freq=A, rot=64, flags=0, mag=1.0, T=4, hq=8, hkv=2, d=64, nb=9, dtype=0, ks=1.0, vs=1.0):
    return pk._lib.kv_append_rotary(q_out, so, q, sq, k, sk, v, sv, kc, vc, slots, pos, freq, rot,
                                    flags, mag, T, hq, hkv, d, nb, dtype, ks, vs, None)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), -1), (dict(hq=-1), -1), (dict(hkv=0), -1), (dict(nb=0), -1), (dict(rot=0), -1),
    (dict(rot=80), -1), (dict(flags=2), -1), (dict(mag=float("inf")), -1), (dict(d=72), -3),
    (dict(rot=24), -3), (dict(d=528, sq=9000, so=9000, sk=2000, sv=2000), -3), (dict(dtype=2), -3), (dict(k=None), -1), (dict(q=None), -1),
    (dict(q_out=None), -1), (dict(pos=None), -1), (dict(freq=None), -1), (dict(slots=None), -1),
    (dict(vc=None), -1), (dict(q=P(4104)), -1), (dict(v=P(4098)), -1), (dict(sk=64), -1),
    (dict(sv=132), -1), (dict(sq=504), -1), (dict(so=0), -1), (dict(dtype=1, ks=0.0), -1),
    (dict(dtype=1, vs=float("nan")), -1)])
def test_rotary_append_refused(pk, bad, code):
    """Before anything of CUDA is called."""
    assert rotary(pk, **bad) == code
    assert rotary(pk, T=0) == pk.KV_OK


def lappend(pk, qo=A, ot=512, oh=64, q=A, qt=512, qh=64, latent=A, sl=576, kr=A, sr=576, w=A,
            eps=1e-6, cache=A, slots=A, pos=A, freq=A, flags=0, mag=1.0, T=4, h=8, l=512, r=64, nb=9):
    return pk._lib.kv_latent_append(qo, ot, oh, q, qt, qh, latent, sl, kr, sr, w, eps, cache, slots,
                                    pos, freq, flags, mag, T, h, l, r, nb, None)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), -1), (dict(h=-1), -1), (dict(l=0), -1), (dict(r=0), -1), (dict(nb=0), -1),
    (dict(flags=4), -1), (dict(l=1032), -3), (dict(l=508), -3), (dict(r=24), -3), (dict(r=272), -3),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(latent=None), -1), (dict(kr=None), -1),
    (dict(cache=None), -1), (dict(q=None), -1), (dict(qo=None), -1), (dict(sl=504), -1),
    (dict(sr=63), -1), (dict(qh=32), -1), (dict(oh=60), -1), (dict(qt=448), -1), (dict(ot=504), -1),
    (dict(qh=2 ** 62), -1), (dict(w=P(4100)), -1), (dict(cache=P(4100)), -1),
    (dict(mag=float("nan")), -1)])
def test_latent_append_refused(pk, bad, code):
    assert lappend(pk, **bad) == code
    assert lappend(pk, T=0) == pk.KV_OK


def attend(pk, out=A, q=A, cache=A, nb=9, bt=A, mb=4, ctx=A, starts=A, parents=A, B=2, T=5, n=4,
           h=16, l=512, r=64, scale=0.1, ws=A, wsb=1 << 40):
    return pk._lib.paged_latent_attention(out, q, cache, nb, bt, mb, ctx, starts, parents, B, T, n, h,
                                          l, r, scale, ws, wsb, None)


@pytest.mark.parametrize("bad,code", [
    (dict(B=-1), -1), (dict(T=-1), -1), (dict(n=0), -1), (dict(n=129), -7), (dict(h=0), -1),
    (dict(h=129), -3), (dict(l=384), -3), (dict(r=48), -3), (dict(out=None), -1), (dict(q=None), -1),
    (dict(cache=None), -1), (dict(bt=None), -1), (dict(ctx=None), -1), (dict(ws=None), -1),
    (dict(nb=0), -1), (dict(mb=0), -1), (dict(q=P(4104)), -1), (dict(out=P(4104)), -1),
    (dict(scale=float("nan")), -1), (dict(starts=None), -1), (dict(starts=None, T=2, n=2), -1),
    (dict(T=2 ** 31 - 1), -3), (dict(nb=2 ** 27), -3), (dict(mb=2 ** 28), -3)])
def test_latent_attention_refused(pk, bad, code):
    assert attend(pk, **bad) == code
    assert attend(pk, B=0) == pk.KV_OK and attend(pk, T=0) == pk.KV_OK
    n = ctypes.c_size_t(7)
    assert pk._lib.paged_latent_workspace_bytes(2, 4, 16, 384, 64, ctypes.byref(n)) == -3
    assert pk._lib.paged_latent_workspace_bytes(2, 4, 16, 512, 64, None) == -1


def test_binding_refuses(pk):
    """Wrong shapes, types and places, before the library is called."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i64, i32 = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    freq, ws = torch.zeros(32), torch.zeros(1024, dtype=torch.uint8)
    cache = bf(4, 16, 576)
    with pytest.raises(ValueError, match="device memory"):
        pk.kv_latent_append(None, None, bf(3, 512), bf(3, 64), cache, i64, i64, freq)
    with pytest.raises(ValueError, match="L \\+ R"):
        pk.kv_latent_append(None, None, bf(3, 512), bf(3, 32), cache, i64, i64, freq)
    with pytest.raises(ValueError, match="16"):
        pk.kv_latent_append(None, None, bf(3, 512), bf(3, 64), bf(4, 8, 576), i64, i64, freq)
    with pytest.raises(ValueError, match="device memory"):
        pk.kv_append_rotary(None, None, bf(3, 2, 64), bf(3, 2, 64), bf(4, 2, 16, 64),
                            bf(4, 2, 16, 64), i64, i64, freq)
    with pytest.raises(ValueError, match="16"):
        pk.kv_append_rotary(None, None, bf(3, 2, 64), bf(3, 2, 64), bf(4, 2, 8, 64),
                            bf(4, 2, 8, 64), i64, i64, freq)
    with pytest.raises(ValueError, match="device memory"):
        pk.paged_latent_attention(bf(3, 4, 512), bf(3, 4, 576), cache, i32[None].expand(3, 3),
                                  i32, 0.1, ws)
    with pytest.raises(ValueError, match="L \\+ R"):
        pk.paged_latent_attention(bf(3, 4, 512), bf(3, 4, 544), cache, i32[None].expand(3, 3),
                                  i32, 0.1, ws)
    with pytest.raises(ValueError, match="16"):
        pk.CacheLayers([bf(4, 8, 576)])
    layers = pk.CacheLayers([cache, bf(4, 16, 576)])
    assert (layers.num_kv_heads, layers.head_dim, layers.v_ptrs) == (1, 576, 0)
    with pytest.raises(ValueError, match="16"):
        pk.kv_copy_blocks(bf(4, 8, 576), None, i32, i32)


def test_caches_without_values(pk):
    """kv_copy_blocks and kv_tree_compact: a missing V is a latent cache's, a missing K is not."""
    assert pk._lib.kv_copy_blocks(None, None, A, A, 2, 1, 576, 9, 0, None) == -1
    one = (ctypes.c_void_p * 2)(4096, 4096)
    assert pk._lib.kv_tree_compact(one, None, 2, A, 4, A, A, A, A, 2, 4, 1, 576, 9, 0, None) == -1
    assert pk._lib.kv_tree_compact(None, None, 2, A, 4, A, A, A, A, 2, 4, 1, 576, 9, 0, None) == -1


@pytest.mark.parametrize("heads", [2, 8])
def test_a_missing_v_of_caches_with_several_heads_is_refused(pk, heads):
    """Only a latent cache, of one head, has no V: another's pointer was lost on the way."""
    assert pk._lib.kv_copy_blocks(A, None, A, A, 2, heads, 64, 9, 0, None) == pk.KV_ERR_INVALID_ARG
    assert pk._lib.kv_copy_blocks(A, None, A, A, 0, heads, 64, 9, 0, None) == pk.KV_OK
    two = (ctypes.c_void_p * 2)(4096, 1 << 30)
    assert pk._lib.kv_tree_compact(two, None, 2, A, 4, A, A, A, A, 2, 4, heads, 64, 9, 0,
                                   None) == pk.KV_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(h=2 ** 26, r=64, qh=64, oh=64, qt=2 ** 32, ot=2 ** 32),
    dict(h=2 ** 31 - 1, r=16, qh=16, oh=16, qt=2 ** 36, ot=2 ** 36)])
def test_latent_append_refuses_heads_that_its_indexes_do_not_hold(pk, bad):
    """As kv_append_rotary does: 2^29 elements of a token's heads and more."""
    assert lappend(pk, **bad) == pk.KV_ERR_UNSUPPORTED


@pytest.mark.parametrize("length", [3.0, 10.0, 64.0, 300.0, 1e6, 1e12])
def test_frequencies_by_parts_of_any_length(pk, length):
    """Where pairs that make so many turns are not among the pairs: the first of them is pair 0 at
    least, the second is behind it."""
    d, theta = 32, 10000.0
    i = np.arange(d // 2)
    plain = theta ** (-2.0 * i / d)
    pair = lambda t: d * math.log(length / (t * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), d - 1)
    slow = np.clip((i - lo) / (hi - lo), 0, 1) if hi > lo else (i > lo) * 1.0
    want = plain * (1 - slow) + plain / 4 * slow
    f = pk.rotary_frequencies(d, theta, "parts", 4.0, 1.0, 32.0, length)[0]
    assert (np.abs(f - want) <= half_ulp(want) * (1 + 2.0 ** -20)).all()
