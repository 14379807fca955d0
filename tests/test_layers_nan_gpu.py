"""NaN and infinities in the expert layer of few tokens at a served model's sizes: what
they reach, and that a call with them takes about as long as one without."""
import math

import pytest
import torch

from tests.test_layers_gpu import BF16, DEV, choices, close, layer, moe_inputs

pytestmark = pytest.mark.gpu

E, K, H, F = 64, 8, 2048, 1024


@pytest.fixture(scope="module")
def tmg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as t
    yield t
    t.check()


def inputs(T, E=E, H=H, F=F, k=K, seed=0):
    """The last token alone chooses the last k experts, the others among the rest."""
    x, logits, W1, W2, res = moe_inputs(T, E, H, F, 200 + seed)
    logits[:, -k:] = -math.inf
    logits[-1] = -math.inf
    logits[-1, -k:] = torch.linspace(0, 1, k, device=DEV)
    return x, logits, W1, W2, res


def shortest(call):
    """Microseconds of a call, the least of several rows of ten."""
    call()
    best = math.inf
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    return best


@pytest.mark.parametrize("T", [1, 13, 61])
def test_a_token_of_nan_takes_no_longer(tmg, T):
    """Its NaN is its result, and no product is formed again for it: within a factor of four."""
    x, logits, W1, W2, res = inputs(T)
    call = lambda: tmg.moe_layer(x, logits, W1, W2, K, residual=res)
    clean, want = shortest(call), call()
    x[-1, 5] = math.nan
    got = call()
    assert got[-1].isnan().all() and torch.equal(got[:-1], want[:-1])
    taken = shortest(call)
    tmg.check()
    assert taken < 4 * clean + 50, f"{taken:.0f} us, {clean:.0f} without the NaN"


@pytest.mark.parametrize("T", [2, 13, 61])
def test_experts_of_infinities(tmg, T):
    """All weights of the experts that only the last token chose are infinite: every column of every other
    token's sum meets a zero times infinity, and is formed again from its own experts."""
    x, logits, W1, W2, res = inputs(T)
    call = lambda: tmg.moe_layer(x, logits, W1, W2, K, residual=res)
    clean = shortest(call)
    W2[-K:] = math.inf
    got = call()
    want, err = layer(x[:-1], choices(logits, K, True)[:-1], W1, W2, res[:-1])
    close(got[:-1], want, err)
    assert not got[-1].isfinite().any()
    taken = shortest(call)
    here = res.clone()
    tmg.moe_layer(x, logits, W1, W2, K, residual=here, out=here)
    assert torch.equal(here[:-1], got[:-1])
    tmg.check()
    assert taken < 20 * clean + 50, f"{taken:.0f} us, {clean:.0f} with finite weights"


@pytest.mark.parametrize("H,F,k", [(136, 72, 2), (520, 264, 5), (8, 8, 1), (1032, 1000, 3)])
@pytest.mark.parametrize("T", [3, 17, 64])
def test_some_columns_are_formed_again(tmg, T, H, F, k):
    """An infinity here and there in the last token's experts, rows and columns off the tiles' borders, strided
    and unaligned residual and result, in place."""
    x, logits, W1, W2, _ = inputs(T, 16, H, F, k, T)
    for c in {0, H // 3, H - 1}:
        W2[-1, c, F // 2] = -math.inf
        W2[-k, c, 0] = math.nan
    wide = torch.randn(T, H + 24, generator=torch.Generator().manual_seed(T)).to(BF16).to(DEV)
    for off in (0, 8, 3):
        res = wide[:, off:off + H]
        want, err = layer(x[:-1], choices(logits, k, True)[:-1], W1, W2, res[:-1])
        got = tmg.moe_layer(x, logits, W1, W2, k, residual=res)
        close(got[:-1], want, err)
        hit = {c for c in range(H) if not got[-1, c].isfinite()}
        assert hit == {0, H // 3, H - 1}
        room = wide.clone()
        here = room[:, off:off + H]
        tmg.moe_layer(x, logits, W1, W2, k, residual=here, out=here)
        assert torch.equal(here[:-1], got[:-1])
        assert torch.equal(room[:, :off], wide[:, :off]) and torch.equal(room[:, off + H:], wide[:, off + H:])
        none = tmg.moe_layer(x, logits, W1, W2, k)
        want, err = layer(x[:-1], choices(logits, k, True)[:-1], W1, W2, None)
        close(none[:-1], want, err)
    tmg.check()
