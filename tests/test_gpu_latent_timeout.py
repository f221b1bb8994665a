"""paged_latent_attention after a wait that ran out: what was under way has landed before the
kernel's shared memory is another's."""
import pytest
import torch

from test_gpu_latent import BF, Case, pk  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stall", [1, 1000, 40000])
@pytest.mark.parametrize("bases,counts,H,L,rope", [
    # a range that fits the ring, so that no copy waits for a free place, and one that does not
    ([30], None, 16, 512, 64), ([700, 90], None, 16, 512, 64), ([9000, 20000], None, 16, 512, 64),
    ([100, 40], [3, 1], 20, 256, 32), ([20000], None, 40, 256, 64),
    ([30], None, 128, 512, 64), ([700, 90], None, 128, 512, 64), ([9000, 20000], None, 128, 512, 64),
    ([100, 40], [3, 1], 100, 256, 32), ([20000, 300], [2, 3], 64, 256, 64)])
def test_the_call_behind_one_that_gave_up_is_right(pk, stall, bases, counts, H, L, rope):  # noqa: F811
    """Launched directly behind it, on the same SMs; several times, so that the roles are cut off in
    different places."""
    c = Case(bases, counts, H, L, rope, seed=H + L)
    good = c.run(pk)
    c.check(good)
    ws = pk.alloc_latent_workspace(len(bases), c.max_nodes, H, L, rope)
    i32 = lambda a: torch.from_numpy(a).int().cuda()  # noqa: E731
    args = (c.q.cuda(), c.cache.cuda(), i32(c.bt), i32(c.lens), c.scale, ws)
    kw = dict(node_starts=None if c.single else i32(c.starts), max_nodes=c.max_nodes)
    cut = torch.empty((c.total, H, L), dtype=BF, device="cuda")
    outs = [torch.empty_like(cut) for _ in range(4)]
    torch.cuda.synchronize()
    for out in outs:
        pk.set_pipeline_stall(stall)
        try:
            pk.paged_latent_attention(cut, *args, **kw)
        finally:
            pk.set_pipeline_stall(0)
        pk.paged_latent_attention(out, *args, **kw)
    torch.cuda.synchronize()
    assert pk.get_device_error()[0] == pk.DEVERR_PIPELINE_TIMEOUT
    for out in outs:
        assert torch.equal(out, good)
