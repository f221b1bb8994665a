"""Draft-tree attention and its neighbours on the GPU, at values and shapes where a result
can be lost without a fault: infinities and NaN that a node sees.

Where an output is finite, the tolerances are those of test_gpu_tree.py."""
import numpy as np
import pytest
import torch

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
