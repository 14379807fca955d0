"""The expert layer of few tokens at widths where the second kernel's clusters just fit the
GPU, and just do not."""
import pytest
import torch

from tests.test_layers_gpu import check_layer, moe_inputs
from tests.test_layers_nan_gpu import shortest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tmg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as t
    yield t
    t.check()


@pytest.mark.parametrize("T", [1, 13, 40])
@pytest.mark.parametrize("H", [2440, 3592, 3848, 4480, 4616, 4744, 4872, 7304, 9096, 9216, 9344, 9728, 9736])
def test_widths_around_the_clusters_limits(tmg, T, H):
    x, logits, W1, W2, res = moe_inputs(T, 8, H, 264, 300)
    check_layer(tmg, x, logits, W1, W2, 2, residual=res)


def test_two_more_tiles_take_no_second_turn(tmg):
    """38 column tiles beside 36, the clusters of four that fit at once: 4 % more weights."""
    times = []
    for H in (4608, 4864):
        states = [moe_inputs(13, 32, H, 1024, 310 + i) for i in range(2)]         # 0.8 GB each, more than L2 holds
        turn = lambda: [tmg.moe_layer(x, g, W1, W2, 4) for x, g, W1, W2, _ in states]
        times.append(shortest(turn))
        del states
        torch.cuda.empty_cache()
    tmg.check()
    assert times[1] < 1.15 * times[0], times
