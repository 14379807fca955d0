"""The operators together, as examples/moe_layer.py uses them: a training step
against the same block in 64 bits (torch autograd on the CPU).

Every tensor between two calls is rounded to bfloat16 (2^-8 relative, about
2^-9.5 in the mean square); the longest chain, from dv to the gradient of W1,
has nine such roundings in either direction, so norms agree within
sqrt(18) 2^-9.5 = 0.6 %; twice that is allowed."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def reference(block, x, dv, experts):
    """The block in 64 bits with the given choice of experts."""
    W = torch.float64
    p = {n: getattr(block, n).cpu().to(W).requires_grad_() for n in ("router", "W1", "W2", "Wa", "ba", "Wb", "bb")}
    xx = x.cpu().to(W).requires_grad_()
    logits = xx @ p["router"].T
    w = logits.gather(1, experts).softmax(1)
    F = p["W2"].shape[2]
    u = xx
    for j in range(experts.shape[1]):
        z = torch.einsum("th,tfh->tf", xx, p["W1"][experts[:, j]])
        h = z[:, :F] * torch.sigmoid(z[:, :F]) * z[:, F:]
        u = u + w[:, j, None] * torch.einsum("tf,thf->th", h, p["W2"][experts[:, j]])
    a = torch.nn.functional.gelu(u @ p["Wa"].T + p["ba"])
    v = u + a @ p["Wb"].T + p["bb"]
    v.backward(dv.cpu().to(W))
    return v.detach(), xx.grad, {n: t.grad for n, t in p.items()}


@pytest.mark.parametrize("T,H,F,E,k,A", [(1, 64, 32, 4, 2, 48), (97, 128, 72, 12, 3, 200), (300, 256, 128, 8, 2, 64)])
def test_block_forward_and_backward(T, H, F, E, k, A):
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as tmg
    from examples.moe_layer import MoeBlock
    block = MoeBlock(H, F, E, k, A, seed=T)
    g = torch.Generator().manual_seed(T + 1)
    x, dv = (torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    v, saved = block.forward(x, train=True)
    dx, grads = block.backward(dv, saved)
    tmg.check()
    rv, rdx, rgrads = reference(block, x, dv, saved[2].experts.cpu().long())
    limit = 2 * 18 ** 0.5 * 2.0 ** -9.5

    def near(name, got, want):
        off = (got.cpu().double() - want).norm() / want.norm().clamp(min=1e-30)
        assert off <= limit, f"{name}: off by {off:.2e}"

    near("v", v, rv)
    near("dx", dx, rdx)
    for n, want in rgrads.items():
        near(n, grads[n], want)


def test_serving_step_matches_training_forward():
    """A token alone takes the decode schedules; its result is that of the same
    token in a batch within the roundings above."""
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as tmg
    from examples.moe_layer import MoeBlock
    block = MoeBlock(512, 256, 16, 4, 256, seed=5)
    x = torch.randn(200, 512, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    whole, _ = block.forward(x)
    for t in (0, 77, 199):
        one, _ = block.forward(x[t:t + 1])
        off = (one.float() - whole[t:t + 1].float()).norm() / whole[t].float().norm()
        assert off <= 2 * 18 ** 0.5 * 2.0 ** -9.5
    tmg.check()
