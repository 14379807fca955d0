"""GPU parity of the expert routing (tmg_moe_route, its gradient) and of the
weighted sum of the experts' answers (tmg_moe_combine, its gradient) against
plain 64-bit evaluations.

The plan is whole numbers: equal.  A weight is a quotient of fp32 exponentials
and their sum: within (E + 8) 2^-23 of itself.  A combined value is an fp32 sum
of at most 17 terms, then one bf16 rounding."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, W = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def tmg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as t
    yield t
    t.check()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def reference(x, k, normalize):
    """Loops over the definition, in 64 bits."""
    x = x.to(W).numpy()
    T, E = x.shape
    experts, weights = np.full((T, k), -1), np.zeros((T, k))
    slots = np.full((T, k), -1)
    for t in range(T):
        able = [e for e in range(E) if x[t, e] > -math.inf]
        able.sort(key=lambda e: (-x[t, e], e))
        pick = able[:k]
        if not pick:
            continue
        top = x[t, pick[0]]
        ex = lambda e: 1.0 if x[t, e] == top else math.exp(x[t, e] - top)
        total = sum(ex(e) for e in (pick if normalize else able))
        experts[t, :len(pick)] = pick
        weights[t, :len(pick)] = [ex(e) / total for e in pick]
    counts = np.bincount(experts[experts >= 0], minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    at = offsets[:-1].copy()
    rows = np.full(T * k, -1)
    for t in range(T):
        for j in range(k):
            if experts[t, j] >= 0:
                slots[t, j] = at[experts[t, j]]
                rows[slots[t, j]] = t
                at[experts[t, j]] += 1
    return weights, experts, offsets, rows, slots


def check_route(tmg, x, k, normalize, dx=None):
    r = tmg.moe_route(x.to(DEV) if dx is None else dx, k, normalize=normalize)
    tmg.check()
    w, experts, offsets, rows, slots = reference(x, k, normalize)
    assert np.array_equal(r.experts.cpu().numpy(), experts)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    got = r.weights.cpu().to(W).numpy()
    assert (np.abs(got - w) <= (x.shape[1] + 8) * 2.0 ** -23 * w + 1e-37).all()
    return r


@pytest.mark.parametrize("T", [0, 1, 5, 33, 130, 153, 1000])
@pytest.mark.parametrize("E,k", [(1, 1), (3, 2), (8, 8), (60, 6), (64, 8), (65, 1), (128, 8), (256, 16), (1000, 4)])
@pytest.mark.parametrize("normalize", [True, False])
def test_route(tmg, T, E, k, normalize):
    check_route(tmg, torch.randn(T, E, generator=gen(T + E)), k, normalize)


@pytest.mark.parametrize("normalize", [True, False])
def test_route_bf16_ties(tmg, normalize):
    x = (torch.randn(500, 64, generator=gen(1)) * 2).round().to(BF16)
    check_route(tmg, x, 8, normalize)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_masks_and_extremes(tmg, dtype, normalize):
    x = torch.randn(300, 40, generator=gen(2))
    x[torch.rand(300, 40, generator=gen(3)) < 0.8] = -math.inf      # often fewer than k left
    x[7], x[8, 1:] = -math.inf, -math.inf
    x[9], x[10, 3], x[11] = torch.finfo(dtype).min, torch.finfo(dtype).min, 0.0
    x[12, 5], x[13, 4:6] = math.inf, math.inf
    x[14], x[14, 6], x[14, 9] = -math.inf, -0.0, 0.0
    x[15] = torch.finfo(dtype).max
    check_route(tmg, x.to(dtype), 6, normalize)


def test_route_nan_is_never_chosen(tmg):
    x = torch.randn(50, 16, generator=gen(4))
    masked = x.clone()
    at = torch.rand(50, 16, generator=gen(5)) < 0.3
    x[at], masked[at] = math.nan, -math.inf
    x[3], masked[3] = math.nan, -math.inf
    r, m = tmg.moe_route(x.to(DEV), 4), tmg.moe_route(masked.to(DEV), 4)
    tmg.check()
    for a, b in zip(r, m):
        assert torch.equal(a, b)


def test_route_one_expert_takes_all_and_strides(tmg):
    x = torch.randn(700, 80, generator=gen(6))
    x[:, 11] = 50.0
    check_route(tmg, x[:, 5:69], 1, True, x.to(DEV)[:, 5:69])


def test_route_many_tokens(tmg):
    """Against torch at a size the loops above would not reach."""
    x = torch.randn(70001, 96, generator=gen(7)).to(DEV)
    r = tmg.moe_route(x, 5)
    tmg.check()
    assert torch.equal(r.experts.long(), x.topk(5, dim=1).indices)
    flat = r.experts.reshape(-1).long()
    order = flat.argsort(stable=True)
    assert torch.equal(r.rows.long(), order // 5)
    assert torch.equal(r.slots.reshape(-1)[order].long(), torch.arange(len(flat), device=DEV))
    assert torch.equal(r.offsets[1:].long(), torch.bincount(flat, minlength=96).cumsum(0))


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (77, 60, 6), (300, 200, 8), (40, 700, 3)])
def test_route_backward(tmg, normalize, dtype, T, E, k):
    x = torch.randn(T, E, generator=gen(8))
    if T > 1:
        x[torch.rand(T, E, generator=gen(9)) < 0.5] = -math.inf
        x[3] = -math.inf
    x = x.to(dtype)
    dw = torch.randn(T, k, generator=gen(10))
    r = tmg.moe_route(x.to(DEV), k, normalize=normalize)
    d = tmg.moe_route_backward(x.to(DEV), r.experts, dw.to(DEV), normalize=normalize)
    tmg.check()
    w, experts, _, _, _ = reference(x, k, normalize)
    xs, g = x.to(W).numpy(), np.zeros((T, E))
    for t in range(T):
        pick = experts[t][experts[t] >= 0]
        if not len(pick):
            continue
        n = len(pick)
        mean = (w[t, :n] * dw[t, :n].to(W).numpy()).sum()
        if not normalize:
            able = xs[t] > -math.inf
            e = np.where(able, np.exp(np.where(able, xs[t] - xs[t, pick[0]], 0)), 0)
            g[t] -= e / e.sum() * mean
            mean = 0.0
        g[t, pick] += w[t, :n] * (dw[t, :n].to(W).numpy() - mean)
    # fp32: a few roundings of terms of size w |dw|
    bound = (E + 16) * 2.0 ** -22 * np.abs(dw.numpy()).max(1, keepdims=True) + 1e-30
    if dtype == BF16:
        bound = bound + 2.0 ** -8 * np.abs(g)
    assert (np.abs(d.cpu().to(W).numpy() - g) <= bound).all()


@pytest.mark.parametrize("normalize", [True, False])
def test_route_backward_against_differences(tmg, normalize):
    """Central differences of the weights themselves: step 2^-6, fp32 weights
    off by 2^-20, third-order term h^2."""
    T, E, k, h = 20, 24, 3, 2.0 ** -6
    x = torch.randn(T, E, generator=gen(11))
    dw = torch.randn(T, k, generator=gen(12))
    r = tmg.moe_route(x.to(DEV), k, normalize=normalize)
    d = tmg.moe_route_backward(x.to(DEV), r.experts, dw.to(DEV), normalize=normalize).cpu()
    experts = r.experts.cpu()
    for e in range(E):
        up, down = x.clone(), x.clone()
        up[:, e] += h
        down[:, e] -= h
        ru, rd = (tmg.moe_route(v.to(DEV), k, normalize=normalize) for v in (up, down))
        same = ((ru.experts.cpu() == experts) & (rd.experts.cpu() == experts)).all(1)
        assert same.sum() >= T // 2
        diff = ((ru.weights - rd.weights).cpu() * dw).sum(1) / (2 * h)
        bound = dw.abs().sum(1) * (h * h + 2.0 ** -20 / h)
        assert ((diff - d[:, e]).abs() <= bound)[same].all()
    tmg.check()


# ------------------------------------------------------------------- combine

def plan(T, k, R, seed):
    slots = torch.randperm(R, generator=gen(seed))[:T * k].view(T, k).int()
    slots[torch.rand(T, k, generator=gen(seed + 1)) < 0.1] = -1
    if T > 2:
        slots[2] = -1                     # a token with no expert
        slots[0, 0] = R + 5               # outside: adds nothing
    return slots


@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 8, 4096), (37, 2, 200), (130, 6, 1023), (50, 16, 2056), (3, 3, 1), (0, 2, 16)])
@pytest.mark.parametrize("weighted,residual", [(True, True), (True, False), (False, False), (False, True)])
def test_combine(tmg, T, k, H, weighted, residual):
    R = T * k + 3
    Y, w = torch.randn(R, H, generator=gen(20)).to(BF16), torch.rand(T, k, generator=gen(21))
    res, slots = torch.randn(T, H, generator=gen(22)).to(BF16), plan(T, k, R, 23)
    out = tmg.moe_combine(Y.to(DEV), slots.to(DEV), w.to(DEV) if weighted else None,
                          residual=res.to(DEV) if residual else None)
    tmg.check()
    ok = ((slots >= 0) & (slots < R))[..., None]
    terms = Y.to(W)[slots.long().clamp(0, R - 1)] * ok * (w.to(W)[..., None] if weighted else 1.0)
    want = terms.sum(1) + (res.to(W) if residual else 0.0)
    size = terms.abs().sum(1) + (res.to(W).abs() if residual else 0.0)
    assert ((out.cpu().to(W) - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 20 * 2.0 ** -24 * size + 1e-38).all()


def test_combine_strides_and_in_place(tmg):
    T, k, H, R = 40, 4, 96, 200
    Y, X, w = (torch.randn(*s, generator=gen(24)) for s in ((R, H + 9), (T, H + 16), (T, k)))
    Y, X, slots = Y.to(BF16), X.to(BF16), plan(T, k, R, 25)
    dX = X.to(DEV)
    tmg.moe_combine(Y.to(DEV)[:, 1:1 + H], slots.to(DEV), w.to(DEV), residual=dX[:, 8:8 + H], out=dX[:, 8:8 + H])
    tmg.check()
    ok = ((slots >= 0) & (slots < R))[..., None]
    want = (Y[:, 1:1 + H].to(W)[slots.long().clamp(0, R - 1)] * ok * w.to(W)[..., None]).sum(1) + X[:, 8:8 + H].to(W)
    assert torch.allclose(dX[:, 8:8 + H].cpu().to(W), want, rtol=2.0 ** -8, atol=1e-5)
    assert torch.equal(dX[:, :8].cpu(), X[:, :8]) and torch.equal(dX[:, 8 + H:].cpu(), X[:, 8 + H:])


def test_combine_unused_rows_are_not_read(tmg):
    """NaN in rows that no slot names."""
    Y = torch.full((10, 64), math.nan, dtype=BF16)
    Y[4] = 2.0
    slots = torch.tensor([[4, -1], [-1, -1]], dtype=torch.int32)
    out = tmg.moe_combine(Y.to(DEV), slots.to(DEV), torch.tensor([[0.5, math.nan], [1.0, 1.0]], device=DEV))
    tmg.check()
    assert (out[0] == 1.0).all() and (out[1] == 0.0).all()


def test_combine_past_32_bits(tmg):
    """Rows of Y, out and dY beyond 2^31 elements."""
    T, H = 530000, 4096
    Y = torch.zeros((T, H), dtype=BF16, device=DEV)
    Y[T - 40:] = torch.randint(-4, 5, (40, H), generator=gen(40)).to(BF16).to(DEV)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)[:, None].contiguous()
    out = tmg.moe_combine(Y, slots)
    dY, dw = tmg.moe_combine_backward(out, Y, slots)
    tmg.check()
    assert torch.equal(out[T - 50:], Y[T - 50:]) and torch.equal(dY[T - 50:], Y[T - 50:])
    assert torch.equal(dw[T - 50:, 0].cpu().to(W), Y[T - 50:].cpu().to(W).square().sum(1))


@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 8, 4096), (37, 2, 200), (130, 6, 1023), (20, 16, 5000), (3, 3, 1), (0, 2, 16)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_backward(tmg, T, k, H, weighted):
    R = T * k + 3
    Y, w = torch.randn(R, H, generator=gen(26)).to(BF16), torch.rand(T, k, generator=gen(27))
    d, slots = torch.randn(T, H, generator=gen(28)).to(BF16), plan(T, k, R, 29)
    dY, dw = tmg.moe_combine_backward(d.to(DEV), Y.to(DEV), slots.to(DEV), w.to(DEV) if weighted else None)
    tmg.check()
    ok = (slots >= 0) & (slots < R)
    y = Y.to(W)[slots.long().clamp(0, R - 1)] * ok[..., None]
    prod = y * d.to(W)[:, None]
    assert ((dw.cpu().to(W) - prod.sum(2)).abs() <= (H + 8) * 2.0 ** -24 * prod.abs().sum(2) + 1e-38).all()
    want = (d.to(W)[:, None] * (w.to(W)[..., None] if weighted else 1.0)).expand(T, k, H)[ok]
    got = dY.cpu().to(W)[slots.long()[ok]]
    assert ((got - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 1e-38).all()


def test_combine_backward_against_differences(tmg):
    """Along a direction of Y and one of the weights, against differences of
    the 64-bit sum."""
    T, k, H = 12, 3, 40
    Y, w = torch.randn(T * k, H, generator=gen(30)).to(BF16), torch.rand(T, k, generator=gen(31))
    d, slots = torch.randn(T, H, generator=gen(32)).to(BF16), torch.randperm(T * k, generator=gen(33)).view(T, k).int()
    dY, dw = tmg.moe_combine_backward(d.to(DEV), Y.to(DEV), slots.to(DEV), w.to(DEV))
    tmg.check()
    loss = lambda y, v: ((v[..., None] * y[slots.long()]).sum(1) * d.to(W)).sum()
    vy, vw, h = torch.randn(T * k, H, dtype=W, generator=gen(34)), torch.randn(T, k, dtype=W, generator=gen(35)), 1e-3
    y, v = Y.to(W), w.to(W)
    dy, dwc = dY.cpu().to(W), dw.cpu().to(W)
    assert abs((dwc * vw).sum() - (loss(y, v + h * vw) - loss(y, v - h * vw)) / (2 * h)) <= 1e-4 * (dwc * vw).norm()
    assert abs((dy * vy).sum() - (loss(y + h * vy, v) - loss(y - h * vy, v)) / (2 * h)) <= 6 * 2.0 ** -9 * (dy * vy).norm()


def test_route_refusals(tmg):
    x = torch.zeros(4, 8, device=DEV)
    r = tmg.moe_route(x, 2)
    Y = torch.zeros(8, 16, dtype=BF16, device=DEV)
    for call in (lambda: tmg.moe_route(x, 0), lambda: tmg.moe_route(x, 9), lambda: tmg.moe_route(x[:, :0], 1),
                 lambda: tmg.moe_route(torch.zeros(2, 1025, device=DEV), 1),
                 lambda: tmg.moe_route(torch.zeros(2, 64, device=DEV), 17)):
        with pytest.raises(tmg.TmgError):
            call()
    with pytest.raises(TypeError):
        tmg.moe_route(x.half(), 2)
    for call in (lambda: tmg.moe_route(x.T.contiguous().T, 2), lambda: tmg.moe_route(x[0], 2), lambda: tmg.moe_route(x.cpu(), 2),
                 lambda: tmg.moe_route_backward(x, r.experts.long(), r.weights),
                 lambda: tmg.moe_route_backward(x, r.experts, r.weights[:2]),
                 lambda: tmg.moe_combine(Y.float(), r.slots, r.weights),
                 lambda: tmg.moe_combine(Y, r.slots.long(), r.weights),
                 lambda: tmg.moe_combine(Y, r.slots, r.weights, residual=Y),
                 lambda: tmg.moe_combine_backward(Y, Y, r.slots, r.weights)):
        with pytest.raises(ValueError):
            call()
    tmg.check()
