"""The README's Python examples run, one after the other, as they are written there."""
import os
import re

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("fork", [False, True])
def test_the_readme_examples_run(fork):
    """With `fork`, sequence 0 has become a branch of sequence 1 between them: the tail block
    that they share is copied before the tree's tokens go to it."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    assert len(blocks) == 2
    ns = {}
    exec(blocks[0], ns)
    alloc, pk, first_k = ns["alloc"], ns["pk"], ns["k_new"]
    if fork:
        alloc.free(0)
        alloc.fork(1, 0, 1)
    exec(blocks[1], ns)
    torch.cuda.synchronize()
    assert pk.get_device_error()[0] == 0
    assert len(ns["cow_src"]) == (1 if fork else 0)
    accepted = ns["accept_lens"].cpu().numpy()
    assert (accepted >= 1).all() and torch.isfinite(ns["out"].float()).all()
    lens = [r["len"] for r in alloc.trace([0, 1])]
    assert lens == list(1 + accepted)
    # the committed token, then the accepted nodes' keys, in each sequence's own blocks
    k, starts, nodes = ns["k_cache"], ns["starts"].cpu().numpy(), ns["accept_nodes"].cpu().numpy()
    bt = ns["bt"].cpu().numpy()
    for s in range(2):
        assert torch.equal(k[bt[s, 0], :, 0], first_k[1 if fork else s])
        for i in range(accepted[s]):
            assert torch.equal(k[bt[s, 0], :, 1 + i], ns["k_new"][starts[s] + nodes[s, i]])
    assert np.unique(bt[:, 0]).size == 2
