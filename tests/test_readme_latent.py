"""The README's example of rotary positions and a latent cache runs as it is written there."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_latent_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```py\n(.*?)```", f.read(), re.S)
    assert len(blocks) == 1
    ns = {}
    exec(blocks[0], ns)
    torch.cuda.synchronize()
    assert ns["pk"].get_device_error()[0] == 0
    assert torch.isfinite(ns["out"].float()).all() and (ns["out"] != 0).any()
    assert [r["len"] for r in ns["alloc"].trace([0, 1])] == [3, 3]
    # the row of the last step: its latent has a mean square of one
    row = ns["cache"][int(ns["bt"][1, 0]), 2].float()
    assert abs(float((row[:512] ** 2).mean()) - 1) < 0.01
    assert (ns["k_cache"][0, :, 0] != 0).any() and (ns["k_cache"][0, :, 1:] == 0).all()
