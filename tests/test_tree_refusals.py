"""Draft-tree calls on the CPU: what they refuse, and how."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build_native()
    import paged_kv_cache_21_gb300 as pk
    return pk


NO_MEMORY = """
import resource, sys
import numpy as np
import paged_kv_cache_21_gb300 as pk
a = pk.BlockAllocator(8, 1, 64)
a.add(0, 20)
before = (a.trace(), a.stats())
ids, counts, lens = np.zeros(4, np.int64), np.ones(4, np.int32), np.zeros(4, np.int64)
out = np.zeros(64, np.int64)
p = lambda x: x.ctypes.data
# room for a table of 2^30 rows (8 GB) there is not: the call ends before it reads them
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (1 << 28), resource.RLIM_INFINITY))
n = 1 << 30
step = pk._lib.kv_tree_step(a._h, p(ids), p(counts), n, p(out), p(out), 4, p(out), p(out), p(out),
                            p(out), 4, None)
cut = pk._lib.kv_seq_truncate(a._h, p(ids), p(lens), n)
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
assert (a.trace(), a.stats()) == before
print(step, cut)
"""


def test_a_failed_host_allocation_has_a_code_of_its_own(pk):
    r = subprocess.run([sys.executable, "-c", NO_MEMORY], cwd=ROOT, capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == [str(pk.KV_ERR_OUT_OF_MEMORY)] * 2


@pytest.mark.parametrize("block", [8, 15, 32])
def test_caches_of_other_blocks_are_refused(pk, block):
    """Blocks of 16 tokens are what the kernels address: with 8 they would read behind the
    cache's end."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    kc = torch.zeros((4, 2, block, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="16"):
        pk.paged_tree_attention(torch.empty_like(q), q, kc, kc, i32(1, 2), i32(1), i32(2), i32(3), 3,
                                0.1, torch.zeros(1024, dtype=torch.uint8))
    with pytest.raises(ValueError, match="16"):
        pk.CacheLayers([kc], [kc])
