"""Routing at the largest number of (token, choice) pairs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def tmg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as t
    yield t
    t.check()


def test_route_pairs_just_below_2_31(tmg):
    """Every token takes all 16 experts, so token t's row of expert e is e T + t;
    T k = 2^31 - 16, and the plan's last block has 112 pairs."""
    k, T = 16, 2 ** 31 // 16 - 1
    logits = torch.empty((T, k), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    step = 1 << 23
    for t0 in range(0, T, step):
        n = min(step, T - t0)
        logits[t0:t0 + n] = torch.rand(n, k, generator=g, device=DEV).to(torch.bfloat16)
    r = tmg.moe_route(logits, k)
    tmg.check()
    assert torch.equal(r.offsets.long().cpu(), torch.arange(k + 1) * T)
    for t0 in list(range(0, T, 16 * step)) + [T - 1000]:
        n = min(step, T - t0)
        e, t = r.experts[t0:t0 + n].long(), torch.arange(t0, t0 + n, device=DEV)
        assert torch.equal(e, logits[t0:t0 + n].float().sort(dim=1, descending=True, stable=True).indices)
        assert torch.equal(r.slots[t0:t0 + n].long(), e * T + t[:, None])
    tail = torch.arange(T - 5000, T, device=DEV)
    for e in range(k):
        assert torch.equal(r.rows[e * T + T - 5000:e * T + T].long(), tail)
        assert torch.equal(r.rows[e * T:e * T + 5000].long(), torch.arange(5000, device=DEV))
    del r, logits
    torch.cuda.empty_cache()
