"""GPU parity of the whole expert layer (tmg_moe_layer) and of the dense product with
low-rank adapters (tmg_lora_linear and its gradients) against plain 64-bit
evaluations.

Bounds, from the arithmetic: a product of K terms with S = sum |a b| is off by at
most K 2^-22 S (fp32 sums in any order, with slack for the tensor core's alignment of
addends); a rounding to bf16 by 2^-8 of the value; weights, scales and activations
by 2^-16 of theirs.  What is rounded between two products (the experts' hidden values,
their answers before the weighted sum, u and dU) carries its error through the
second one's |operand|.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
W = torch.float64
SUM, ROUND, SOFT = 2.0 ** -22, 2.0 ** -8, 2.0 ** -16


@pytest.fixture(scope="module")
def tmg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as t
    yield t
    t.check()


def normal(shape, seed, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).to(DEV)


def close(got, want, err, name=""):
    assert torch.isfinite(got).all(), name
    off, bound = (got.to(W) - want).abs(), err + ROUND * 1.01 * (want.abs() + err) + 1e-30
    worst = (off / bound).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{name} off by {worst:.3g} of the bound"


# ------------------------------------------------------------- the expert layer

def choices(logits, k, normalize):
    """(T, E) weights of the chosen experts, zeros elsewhere, by the definition."""
    x = logits.double().cpu()
    w = torch.zeros_like(x)
    for t, row in enumerate(x.tolist()):
        able = [e for e in range(len(row)) if row[e] > -math.inf]
        chosen = sorted(able, key=lambda e: (-row[e], e))[:k]
        if not chosen:
            continue
        top = row[chosen[0]]
        ex = {e: 1.0 if row[e] == top else math.exp(row[e] - top) for e in able}
        total = sum(ex[e] for e in (chosen if normalize else able))
        for e in chosen:
            w[t, e] = ex[e] / total
    return w.to(DEV)


def layer(x, w, W1, W2, residual):
    """out in 64 bits and its error bound before the last rounding."""
    T, H = x.shape
    F = W2.shape[2]
    out = residual.to(W).clone() if residual is not None else torch.zeros(T, H, dtype=W, device=DEV)
    err = torch.zeros_like(out)
    for e in range(w.shape[1]):
        t = (w[:, e] != 0).nonzero()[:, 0]
        if not len(t):
            continue
        a, b1, b2 = x[t].to(W), W1[e].to(W), W2[e].to(W)
        z, ez = a @ b1.T, H * SUM * (a.abs() @ b1.abs().T)
        g, up = z[:, :F], z[:, F:]
        silu = g * torch.sigmoid(g)
        h = silu * up
        eh = 1.1 * ez[:, :F] * up.abs() + silu.abs() * ez[:, F:] + 1.1 * ez[:, :F] * ez[:, F:] + SOFT * (h.abs() + up.abs())
        eh = eh + ROUND * 1.01 * (h.abs() + eh)
        y = h @ b2.T
        ey = eh @ b2.abs().T + (F + 16) * SUM * ((h.abs() + eh) @ b2.abs().T)
        ey = ey + ROUND * 1.01 * (y.abs() + ey)
        out[t] += w[t, e, None] * y
        err[t] += w[t, e, None] * (ey + SOFT * y.abs())
    return out, err + 32 * SUM * out.abs()


def moe_inputs(T, E, H, F, seed=0, dtype=F32):
    return (normal((T, H), seed), normal((T, E), seed + 1, dtype=dtype), normal((E, 2 * F, H), seed + 2, H ** -0.5),
            normal((E, H, F), seed + 3, F ** -0.5), normal((T, H), seed + 4))


def check_layer(tmg, x, logits, W1, W2, k, normalize=True, residual=None, name="", **more):
    got = tmg.moe_layer(x, logits, W1, W2, k, normalize=normalize, residual=residual, **more)
    tmg.check()
    close(got, *layer(x, choices(logits, k, normalize), W1, W2, residual), name)
    return got


@pytest.mark.parametrize("H,F", [(64, 64), (136, 72), (512, 256), (520, 200), (1032, 264), (130, 70), (8, 8), (257, 33)])
@pytest.mark.parametrize("T", [1, 2, 7, 17, 61])
def test_layer(tmg, T, H, F):
    x, logits, W1, W2, res = moe_inputs(T, 16, H, F)
    check_layer(tmg, x, logits, W1, W2, 4, residual=res)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (8, 1), (33, 8), (64, 16), (128, 8), (256, 4), (300, 8), (1024, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("normalize", [True, False])
def test_layer_routes(tmg, E, k, dtype, normalize):
    for T in (1, 9):
        x, logits, W1, W2, _ = moe_inputs(T, E, 72, 40, 10, dtype)
        check_layer(tmg, x, logits, W1, W2, k, normalize, name=f"T={T}")


@pytest.mark.parametrize("T", [15, 16, 31, 32, 33, 47, 48, 49, 63, 64, 65, 128, 129, 300])
def test_layer_tokens(tmg, T):
    x, logits, W1, W2, res = moe_inputs(T, 24, 264, 136, 20)
    check_layer(tmg, x, logits, W1, W2, 3, residual=res)


@pytest.mark.parametrize("T", [1, 3, 30, 100])
def test_layer_masks(tmg, T):
    """Experts masked off, fewer left than k, tokens without any (out = residual), NaN and equal logits."""
    x, logits, W1, W2, res = moe_inputs(T, 12, 136, 64, 30, BF16)
    logits[torch.rand(T, 12, generator=torch.Generator().manual_seed(31)).to(DEV) < 0.6] = -math.inf
    logits[0] = -math.inf
    if T > 2:
        logits[1] = 0.5
        logits[2, :5] = math.nan
    clean = torch.where(torch.isnan(logits), -math.inf, logits)
    for residual in (res, None):
        got = tmg.moe_layer(x, logits, W1, W2, 4, residual=residual)
        tmg.check()
        close(got, *layer(x, choices(clean, 4, True), W1, W2, residual))
    assert torch.equal(tmg.moe_layer(x, logits, W1, W2, 4, residual=res)[0], res[0])
    logits[:] = -math.inf
    assert torch.equal(tmg.moe_layer(x, logits, W1, W2, 4, residual=res), res)
    assert not tmg.moe_layer(x, logits, W1, W2, 4).any()


def test_layer_infinite_logits(tmg):
    x, logits, W1, W2, _ = moe_inputs(4, 8, 64, 64, 40)
    logits[0, 3] = logits[0, 5] = math.inf
    logits[1, 2] = math.inf
    logits[2] = torch.finfo(F32).min
    logits[3, :7] = torch.finfo(F32).min
    for normalize in (True, False):
        check_layer(tmg, x, logits, W1, W2, 3, normalize)


@pytest.mark.parametrize("T", [2, 20, 64, 90])
def test_layer_keeps_tokens_apart(tmg, T):
    """NaN and infinities in a token, or in the weights of experts that only it chose, reach no other token."""
    E = 10
    x, logits, W1, W2, res = moe_inputs(T, E, 264, 136, 50)
    logits[:, :2] = -math.inf
    bad = T - 1
    logits[bad] = -math.inf
    logits[bad, :2] = 1.0
    for value in (math.nan, math.inf):
        for spoil in ("x", "W1", "W2", "both"):
            a, b1, b2 = x.clone(), W1.clone(), W2.clone()
            if spoil == "x":
                a[bad, 7] = value
            if spoil in ("W1", "both"):
                b1[0, 3, 5] = value
            if spoil in ("W2", "both"):
                b2[1, 200, 100] = value
            got = tmg.moe_layer(a, logits, b1, b2, 2, residual=res)
            tmg.check()
            want, err = layer(x, choices(logits, 2, True), W1, W2, res)
            close(got[:bad], want[:bad], err[:bad], f"{spoil} {value}")
            hit = ~torch.isfinite(got[bad])
            assert hit[200] if spoil == "W2" else hit.any(), (spoil, value)
            if spoil == "W2":
                assert hit.sum() == 1


def test_layer_strides_and_in_place(tmg):
    T, E, H, F = 19, 16, 264, 136
    wide = normal((T, H + 40), 60)
    _, _, W1, W2, _ = moe_inputs(T, E, H, F, 61)
    logits = normal((T, E + 5), 62, dtype=F32)[:, :E]
    for x, res in ((wide[:, :H], wide[:, 16:16 + H]), (wide[:, 1:H + 1], wide[:, 3:H + 3]), (wide[:1, :H].expand(T, H), wide[:, :H])):
        out = torch.full((T, H + 24), 5.0, dtype=BF16, device=DEV)
        got = check_layer(tmg, x, logits, W1, W2, 4, residual=res, out=out[:, 8:8 + H])
        assert got.data_ptr() == out[:, 8:].data_ptr() and (out[:, :8] == 5).all() and (out[:, 8 + H:] == 5).all()
    here = wide[:, :H].clone()
    want = tmg.moe_layer(wide[:, :H], logits, W1, W2, 4, residual=here)
    tmg.moe_layer(wide[:, :H], logits, W1, W2, 4, residual=here, out=here)
    assert torch.equal(here, want)


@pytest.mark.parametrize("T", [1, 40, 100])
def test_layer_repeats_bit_for_bit(tmg, T):
    x, logits, W1, W2, res = moe_inputs(T, 32, 1024, 512, 70)
    want = tmg.moe_layer(x, logits, W1, W2, 8, residual=res)
    for _ in range(20):
        assert torch.equal(tmg.moe_layer(x, logits, W1, W2, 8, residual=res), want)
    tmg.check()


def test_layer_of_a_large_model(tmg):
    for T, E, k, H, F in ((1, 64, 8, 2048, 1024), (13, 32, 4, 4096, 2048), (61, 64, 8, 2048, 1024), (5, 8, 2, 4096, 8192)):
        x, logits, W1, W2, res = moe_inputs(T, E, H, F, 80)
        check_layer(tmg, x, logits, W1, W2, k, residual=res, name=str((T, E, k, H, F)))


def test_layer_nothing_to_do(tmg):
    x, logits, W1, W2, res = moe_inputs(3, 4, 64, 32, 90)
    assert tmg.moe_layer(x[:0], logits[:0], W1, W2, 2).shape == (0, 64)
    empty = torch.empty(4, 0, 64, dtype=BF16, device=DEV)
    assert torch.equal(tmg.moe_layer(x, logits, empty, empty.transpose(1, 2).contiguous(), 2, residual=res), res)
    tmg.check()


def test_layer_refuses(tmg):
    x, logits, W1, W2, res = moe_inputs(3, 4, 64, 32, 95)
    for bad in (dict(x=x.half()), dict(x=x.t()), dict(logits=logits.half()), dict(logits=logits[:2]), dict(W1=W1[:, :32]),
                dict(W1=W1.transpose(1, 2)), dict(W2=W2[:3]), dict(residual=res[:, :32]), dict(out=res[:2]), dict(x=x.cpu()),
                dict(k=0), dict(k=5), dict(k=17), dict(W2=W2.float())):
        a = dict(x=x, logits=logits, W1=W1, W2=W2, k=2)
        a.update(bad)
        with pytest.raises((ValueError, TypeError, tmg.TmgError)):
            tmg.moe_layer(**a)


# ------------------------------------------------------------- adapters

def ids_of(kind, M, L, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        i = torch.full((M,), L - 1)
    elif kind == "none":
        i = torch.full((M,), -1)
    elif kind == "each":                                # a request each
        i = torch.randint(-1, L, (M,), generator=g)
    elif kind == "outside":
        i = torch.randint(-1, L, (M,), generator=g)
        i[::3] = L
        i[1::5] = -2 ** 31
        i[2::7] = 2 ** 31 - 1
    else:                                               # requests of some rows each
        n = torch.randint(1, 120, (M,), generator=g)
        i = torch.randint(-1, L, (M,), generator=g).repeat_interleave(n)[:M]
    return i.to(torch.int32).to(DEV)


def lora_inputs(M, N, K, r, L, seed=0):
    return dict(x=normal((M, K), seed), W=normal((N, K), seed + 1, max(K, 1) ** -0.5), A=normal((L, r, K), seed + 2, max(K, 1) ** -0.5),
                B=normal((L, N, r), seed + 3, r ** -0.5), scales=(0.5 + torch.rand(L, generator=torch.Generator().manual_seed(seed))).to(DEV))


def adapted(x, W_, A, B, ids, scales=None, bias=None, residual=None):
    """D, u in 64 bits and the error bounds of both."""
    (M, K), (N, r) = x.shape, B.shape[1:]
    X, Wd = x.to(W), W_.to(W)
    D, err = X @ Wd.T, (K + 8) * SUM * (X.abs() @ Wd.abs().T)
    u, eu = torch.zeros(M, r, dtype=W, device=DEV), torch.zeros(M, r, dtype=W, device=DEV)
    for l in range(A.shape[0]):
        m = (ids == l).nonzero()[:, 0]
        if not len(m):
            continue
        s = 1.0 if scales is None else float(scales[l])
        a, b = A[l].to(W), B[l].to(W)
        u[m] = s * (X[m] @ a.T)
        eu[m] = abs(s) * (K + 8) * SUM * (X[m].abs() @ a.abs().T)
        e = eu[m] + ROUND * 1.01 * (u[m].abs() + eu[m])
        D[m] += u[m] @ b.T
        err[m] += e @ b.abs().T + (r + 8) * SUM * ((u[m].abs() + e) @ b.abs().T)
    if bias is not None:
        D, err = D + bias.to(W), err + SUM * bias.to(W).abs()
    if residual is not None:
        D, err = D + residual.to(W), err + SUM * residual.to(W).abs()
    return D, err + 4 * SUM * D.abs(), u, eu


def check_lora(tmg, t, ids, bias=None, residual=None, scaled=True, name="", **more):
    scales = t["scales"] if scaled else None
    u = torch.empty(len(ids), t["A"].shape[1], dtype=BF16, device=DEV)
    D = tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], ids, scales=scales, bias=bias, residual=residual, u=u, **more)
    plain = tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], ids, scales=scales, bias=bias, residual=residual)
    tmg.check()
    want, err, wu, eu = adapted(t["x"], t["W"], t["A"], t["B"], ids, scales, bias, residual)
    close(D, want, err, name + " D")
    close(u, wu, eu, name + " u")
    assert torch.equal(plain, D), name
    return D, u


def gradients(dD, x, W_, A, B, ids, u, scales=None):
    """(dx, dA, dB) in 64 bits with their error bounds."""
    (M, N), K, r = dD.shape, x.shape[1], A.shape[1]
    d, X, Wd = dD.to(W), x.to(W), W_.to(W)
    dx, ex = d @ Wd, (N + 8) * SUM * (d.abs() @ Wd.abs())
    out = [torch.zeros(A.shape, dtype=W, device=DEV) for _ in range(2)] + [torch.zeros(B.shape, dtype=W, device=DEV) for _ in range(2)]
    dA, eA, dB, eB = out
    for l in range(A.shape[0]):
        m = (ids == l).nonzero()[:, 0]
        if not len(m):
            continue
        s = 1.0 if scales is None else float(scales[l])
        a, b, ul = A[l].to(W), B[l].to(W), u[m].to(W)
        dU, eU = s * (d[m] @ b), abs(s) * (N + 8) * SUM * (d[m].abs() @ b.abs())
        eU = eU + ROUND * 1.01 * (dU.abs() + eU)
        dx[m] += dU @ a
        ex[m] += eU @ a.abs() + (r + 8) * SUM * ((dU.abs() + eU) @ a.abs())
        n = (len(m) + 72) * SUM
        dA[l], eA[l] = dU.T @ X[m], eU.T @ X[m].abs() + n * ((dU.abs() + eU).T @ X[m].abs())
        dB[l], eB[l] = d[m].T @ ul, n * (d[m].abs().T @ ul.abs())
    return (dx, ex + 4 * SUM * dx.abs()), (dA, eA), (dB, eB)


def check_grads(tmg, t, ids, dD, u, scaled=True, name=""):
    scales = t["scales"] if scaled else None
    got = tmg.lora_linear_backward(dD, t["x"], t["W"], t["A"], t["B"], ids, u, scales=scales)
    tmg.check()
    for g, (want, err), n in zip(got, gradients(dD, t["x"], t["W"], t["A"], t["B"], ids, u, scales), ("dx", "dA", "dB")):
        assert g.shape == want.shape and g.is_contiguous()
        close(g, want, err, f"{name} {n}")
    return got


SHAPES = [(64, 64), (136, 264), (520, 1032), (1000, 200), (24, 8), (257, 130), (72, 1001), (1, 64)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("M", [1, 16, 61, 65, 300])
def test_lora(tmg, M, N, K):
    t = lora_inputs(M, N, K, 16, 5)
    for kind in ("runs", "each"):
        check_lora(tmg, t, ids_of(kind, M, 5, M), name=kind)


@pytest.mark.parametrize("r", [1, 3, 4, 8, 12, 16, 24, 40, 64, 72, 128, 136, 256])
@pytest.mark.parametrize("M", [5, 64, 200])
def test_lora_ranks(tmg, r, M):
    t = lora_inputs(M, 264, 328, r, 3, 10)
    check_lora(tmg, t, ids_of("runs", M, 3, r), bias=normal(264, 14, dtype=F32), residual=normal((M, 264), 15))


@pytest.mark.parametrize("kind", ["one", "none", "each", "outside", "runs"])
@pytest.mark.parametrize("M", [3, 33, 63, 64, 128, 129, 255, 257, 513, 900])
def test_lora_requests(tmg, kind, M):
    t = lora_inputs(M, 392, 256, 16, 40, 20)
    check_lora(tmg, t, ids_of(kind, M, 40, M), scaled=M % 2 == 0)


def test_lora_many_adapters(tmg):
    t = lora_inputs(600, 136, 128, 8, 1024, 25)
    check_lora(tmg, t, ids_of("each", 600, 1024, 1))
    check_grads(tmg, t, ids_of("each", 600, 1024, 1), normal((600, 136), 26), normal((600, 8), 27))


@pytest.mark.parametrize("M", [7, 60, 400])
def test_lora_strides_and_in_place(tmg, M):
    N, K = 264, 200
    t = lora_inputs(M, N, K, 16, 4, 30)
    wide, wW = normal((M, K + 56), 31), normal((N, K + 24), 32, 0.1)
    ids = ids_of("runs", M, 4, 5)
    for off in (0, 8, 3):
        t["x"], t["W"] = wide[:, off:off + K], wW[:, off:off + K]
        rwide, D = normal((M, N + 40), 33), torch.full((M, N + 24), 5.0, dtype=BF16, device=DEV)
        check_lora(tmg, t, ids, residual=rwide[:, off:off + N], D=D[:, off:off + N])
        assert (D[:, :off] == 5).all() and (D[:, off + N:] == 5).all()
    here = normal((M, N), 34)
    want = tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], ids, residual=here)
    tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], ids, here, residual=here)
    assert torch.equal(here, want)


@pytest.mark.parametrize("K", [448, 512, 520, 1024, 2056, 4096, 8200])
@pytest.mark.parametrize("M,r", [(1, 1), (1, 8), (1, 16), (1, 20), (1, 32), (2, 16), (3, 5), (4, 8), (5, 6), (32, 1), (33, 1), (3, 16)])
def test_lora_of_few_ranks(tmg, M, r, K):
    """Up to 32 ranks of all rows, where one kernel does it all, and just above."""
    N = 300
    t = lora_inputs(M, N, K, r, 6, 35)
    wide = normal((M, K + 24), 36)
    for off, kind in ((0, "each"), (8, "outside"), (3, "runs")):
        t["x"] = wide[:, off:off + K]
        ids = ids_of(kind, M, 6, K)
        _, u = check_lora(tmg, t, ids, bias=normal(N, 37, dtype=F32), residual=normal((M, N), 38), scaled=off > 0, name=kind)
        room = torch.full((M * r + 2,), 7.0, dtype=BF16, device=DEV)
        tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], ids, scales=t["scales"] if off else None, u=room[1:-1].view(M, r))
        assert torch.equal(room[1:-1].view(M, r), u) and room[0] == 7 and room[-1] == 7


@pytest.mark.parametrize("r", [16, 24])
def test_lora_of_few_ranks_keeps_requests_apart(tmg, r):
    """Infinities of an adapter and of a row reach the rows that have them alone."""
    N, K = 264, 2048
    t = lora_inputs(2, N, K, r, 3, 39)
    ids = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    want = tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], ids)
    t["A"][1], t["B"][1] = float("inf"), float("nan")
    assert torch.equal(tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], ids), want)
    t["A"][2, 1, K - 1] = float("inf")
    got = tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], ids)
    assert torch.equal(got[0], want[0]) and not got[1].isfinite().any()


def test_lora_of_few_ranks_in_a_row(tmg):
    """Calls that read the results of the ones before, in one stream and in a graph."""
    H = 1024
    t = [lora_inputs(2, H, H, 16, 4, 40 + i) for i in range(6)]
    ids = ids_of("each", 2, 4, 1)
    first = t[0]["x"].clone()

    def chain(sync):
        x = first
        for c in t + t:
            x = tmg.lora_linear(x, c["W"], c["A"], c["B"], ids, residual=x)
            if sync:
                torch.cuda.synchronize()
        return x

    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain(False)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = chain(False)
        first.copy_(t[1]["x"])
        graph.replay()
    s.synchronize()
    assert torch.equal(out, chain(True)) and not torch.equal(out, want)
    tmg.check()


@pytest.mark.parametrize("M", [4, 50, 64, 300])
def test_lora_keeps_requests_apart(tmg, M):
    """NaN and infinities of one request, or of its adapter, reach no other request's rows or gradients."""
    N, K, L = 264, 328, 6
    t = lora_inputs(M, N, K, 16, L, 40)
    ids = ids_of("runs" if M > 64 else "each", M, L - 1, 41)
    ids[M // 2] = L - 1
    ids[M // 3] = -1
    others = ids != L - 1
    dD, u = normal((M, N), 44), normal((M, 16), 45)
    want, err, _, _ = adapted(t["x"], t["W"], t["A"], t["B"], ids, t["scales"])
    grads = gradients(dD, t["x"], t["W"], t["A"], t["B"], ids, u, t["scales"])
    for value in (math.nan, math.inf):
        for spoil in ("x", "A", "B", "dD", "u"):
            s = {k: v.clone() for k, v in t.items()}
            d, su = dD.clone(), u.clone()
            if spoil == "x":
                s["x"][M // 2, 5] = value
            elif spoil == "A":
                s["A"][L - 1, 3, 7] = value
            elif spoil == "B":
                s["B"][L - 1, 9, 2] = value
            elif spoil == "dD":
                d[M // 2, 11] = value
            else:
                su[M // 2, 1] = value
            got = tmg.lora_linear(s["x"], s["W"], s["A"], s["B"], ids, scales=s["scales"])
            dx, dA, dB = tmg.lora_linear_backward(d, s["x"], s["W"], s["A"], s["B"], ids, su, scales=s["scales"])
            tmg.check()
            close(got[others], want[others], err[others], f"{spoil} {value} D")
            close(dx[others], *(g[others] for g in grads[0]), f"{spoil} {value} dx")
            close(dA[:L - 1], *(g[:L - 1] for g in grads[1]), f"{spoil} {value} dA")
            close(dB[:L - 1], *(g[:L - 1] for g in grads[2]), f"{spoil} {value} dB")
            if spoil in ("x", "A"):
                assert not torch.isfinite(got[M // 2]).all()
            if spoil == "B":
                assert not torch.isfinite(got[M // 2, 9]) and torch.isfinite(got[M // 2, 10:]).all()


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("M", [1, 60, 200])
def test_lora_gradients(tmg, M, N, K):
    t = lora_inputs(M, N, K, 16, 5, 50)
    for kind in ("runs", "each"):
        check_grads(tmg, t, ids_of(kind, M, 5, M), normal((M, N), 54), normal((M, 16), 55), name=kind)


@pytest.mark.parametrize("r", [1, 3, 4, 8, 12, 16, 24, 40, 64, 72, 128, 136, 256])
def test_lora_gradients_ranks(tmg, r):
    for M in (5, 200):
        t = lora_inputs(M, 264, 328, r, 3, 60)
        check_grads(tmg, t, ids_of("runs", M, 3, r), normal((M, 264), 64), normal((M, r), 65), scaled=r % 2 == 0, name=str(M))


@pytest.mark.parametrize("kind", ["one", "none", "each", "outside", "runs"])
@pytest.mark.parametrize("M", [3, 64, 129, 257, 900])
def test_lora_gradients_requests(tmg, kind, M):
    t = lora_inputs(M, 392, 256, 16, 12, 70)
    check_grads(tmg, t, ids_of(kind, M, 12, M), normal((M, 392), 74), normal((M, 16), 75))


@pytest.mark.parametrize("rows", [1, 64, 65, 128, 130, 192, 257])
def test_lora_gradients_of_few_rows_among_many(tmg, rows):
    """Fewer blocks of rows with an adapter than runs that share the work."""
    M = 2900
    t = lora_inputs(M, 136, 264, 16, 5, 76)
    ids = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    ids[1000:1000 + rows] = 3
    ids[2000:2000 + rows // 2] = 1
    check_grads(tmg, t, ids, normal((M, 136), 77), normal((M, 16), 78))
    ids[2000:2000 + rows // 2] = -1
    check_grads(tmg, t, ids, normal((M, 136), 77), normal((M, 16), 78))


@pytest.mark.parametrize("L", [1, 2, 5, 40])
@pytest.mark.parametrize("M,N,K,r", [(2500, 264, 200, 16), (1500, 520, 136, 64), (700, 1024, 512, 32)])
def test_lora_gradients_in_runs(tmg, M, N, K, r, L):
    """Adapters in one run and cut over several, the factors before dx and after it."""
    t = lora_inputs(M, N, K, r, L, 75)
    for kind in ("runs", "one", "outside"):
        check_grads(tmg, t, ids_of(kind, M, L, L), normal((M, N), 79), normal((M, r), 80), name=kind)


@pytest.mark.parametrize("M,N,K", [(40, 136, 72), (700, 512, 256), (300, 2048, 1000)])
def test_lora_gradients_alone(tmg, M, N, K):
    """Each gradient without the others, and without what only the others need."""
    from tiled_mma_atom_gb300 import _native

    r, L = 16, 3
    t = lora_inputs(M, N, K, r, L, 81)
    ids, d, u = ids_of("runs", M, L, 2), normal((M, N), 82), normal((M, r), 83)
    exact = gradients(d, t["x"], t["W"], t["A"], t["B"], ids, u, t["scales"])
    ptr = lambda x, there: x.data_ptr() if there else 0
    for want in range(8):
        dx, dA, dB = (bool(want >> i & 1) for i in range(3))
        out = [torch.full(shape, 3.0, dtype=BF16, device=DEV) for shape in ((M, K), (L, r, K), (L, N, r))]
        args = _native.pack_lora_grad(d.data_ptr(), ptr(t["x"], dA), ptr(t["W"], dx), ptr(t["A"], dx), ptr(t["B"], dx or dA),
                                      ids.data_ptr(), t["scales"].data_ptr(), ptr(u, dB), ptr(out[0], dx), ptr(out[1], dA),
                                      ptr(out[2], dB), M, N, K, r, L, N, K, K)
        assert _native.lib().tmg_lora_linear_backward(args, torch.cuda.current_stream().cuda_stream) == 0
        tmg.check()
        for i, (g, (w, err)) in enumerate(zip(out, exact)):
            if want >> i & 1:
                close(g, w, err, f"{want} {i}")
            else:
                assert (g == 3).all()


def test_lora_of_a_large_model(tmg):
    for M, N, K, r, L in ((1, 4096, 4096, 16, 8), (16, 8192, 8192, 16, 64), (700, 1024, 4096, 32, 16), (2100, 4096, 2048, 64, 4),
                          (1500, 5000, 4104, 8, 3)):
        t = lora_inputs(M, N, K, r, L, 80)
        ids = ids_of("each" if M < 65 else "runs", M, L, 81)
        _, u = check_lora(tmg, t, ids, residual=normal((M, N), 82), name=str((M, N, K)))
        if M > 64:
            check_grads(tmg, t, ids, normal((M, N), 83), u, name=str((M, N, K)))


@pytest.mark.parametrize("M", [1, 40, 300, 2000])
def test_lora_repeats_bit_for_bit(tmg, M):
    t = lora_inputs(M, 1032, 1024, 16, 6, 90)
    ids, dD, u = ids_of("runs", M, 6, 91), normal((M, 1032), 94), normal((M, 16), 95)
    want = (tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], ids), *tmg.lora_linear_backward(dD, t["x"], t["W"], t["A"], t["B"], ids, u))
    for _ in range(10):
        got = (tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], ids), *tmg.lora_linear_backward(dD, t["x"], t["W"], t["A"], t["B"], ids, u))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    tmg.check()


def test_lora_nothing_to_do(tmg):
    t = lora_inputs(4, 64, 64, 8, 3, 100)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert tmg.lora_linear(t["x"][:0], t["W"], t["A"], t["B"], none).shape == (0, 64)
    dx, dA, dB = tmg.lora_linear_backward(t["x"][:0], t["x"][:0], t["W"], t["A"], t["B"], none,
                                          torch.empty(0, 8, dtype=BF16, device=DEV))
    assert dx.shape == (0, 64) and not dA.any() and not dB.any()
    e = lora_inputs(4, 64, 0, 8, 3, 101)
    bias = normal(64, 102, dtype=F32)
    D = tmg.lora_linear(e["x"], e["W"], e["A"], e["B"], ids_of("each", 4, 3), bias=bias)
    assert torch.equal(D, bias.to(BF16).expand(4, 64))
    n = lora_inputs(4, 0, 64, 8, 3, 103)
    dx, dA, dB = tmg.lora_linear_backward(normal((4, 0), 1), n["x"], n["W"], n["A"], n["B"], ids_of("each", 4, 3), normal((4, 8), 2))
    assert not dx.any() and not dA.any() and dB.shape == (3, 0, 8)
    tmg.check()


def test_lora_refuses(tmg):
    t = lora_inputs(4, 64, 72, 8, 3, 110)
    ids, u, d = ids_of("each", 4, 3), normal((4, 8), 1), normal((4, 64), 2)
    a = dict(x=t["x"], W=t["W"], A=t["A"], B=t["B"], adapters=ids)
    for bad in (dict(x=t["x"].half()), dict(x=t["x"].t().contiguous().t()), dict(W=t["W"][:, :8]), dict(A=t["A"][:, :, :64]),
                dict(A=t["A"][:, :4]), dict(B=t["B"][:2]), dict(adapters=ids.long()), dict(adapters=ids[:3]), dict(adapters=ids.cpu()),
                dict(A=t["A"].transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((ValueError, TypeError, tmg.TmgError)):
            tmg.lora_linear(**{**a, **bad})
        with pytest.raises((ValueError, TypeError, tmg.TmgError)):
            tmg.lora_linear_backward(dD=d, u=u, **{**a, **bad})
    for bad in (dict(scales=t["scales"][:2]), dict(scales=t["scales"].half()), dict(bias=t["scales"]), dict(residual=d[:3]),
                dict(u=u[:, :4]), dict(D=d[:, :32])):
        with pytest.raises((ValueError, TypeError, tmg.TmgError)):
            tmg.lora_linear(**a, **bad)
    big = torch.zeros(1, 257, 72, dtype=BF16, device=DEV)
    with pytest.raises(tmg.TmgError):
        tmg.lora_linear(t["x"], t["W"], big, torch.zeros(1, 64, 257, dtype=BF16, device=DEV), ids)


# ------------------------------------------------------------- together

def test_decoding_step(tmg):
    """A projection with adapters feeding an expert layer, token by token equal to the batch within the bounds,
    eager and replayed from a graph with new inputs."""
    T, E, k, H, F, r, L = 9, 16, 4, 512, 256, 16, 4
    t = lora_inputs(T, H, H, r, L, 120)
    _, logits, W1, W2, _ = moe_inputs(T, E, H, F, 121)
    ids = ids_of("each", T, L, 122)
    x, g, i = t["x"].clone(), logits.clone(), ids.clone()

    def step():
        y = tmg.lora_linear(x, t["W"], t["A"], t["B"], i, scales=t["scales"], residual=x)
        return y, tmg.moe_layer(y, g, W1, W2, k, residual=y)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            captured = step()
    for seed in (0, 1, 2):
        x.copy_(normal((T, H), 130 + seed))
        g.copy_(normal((T, E), 140 + seed, dtype=F32))
        i.copy_(ids_of("each", T, L, 150 + seed))
        graph.replay()
        torch.cuda.synchronize()
        y, out = step()
        assert torch.equal(captured[0], y) and torch.equal(captured[1], out)
        want, err, _, _ = adapted(x, t["W"], t["A"], t["B"], i, t["scales"], None, x)
        close(y, want, err)
        close(out, *layer(y, choices(g, k, True), W1, W2, y))
        for m in range(T):
            one = tmg.lora_linear(x[m:m + 1], t["W"], t["A"], t["B"], i[m:m + 1], scales=t["scales"], residual=x[m:m + 1])
            close(one, want[m:m + 1], err[m:m + 1])
    tmg.check()


@pytest.mark.parametrize("M", [50, 700])
def test_training_step(tmg, M):
    """Forward, loss gradient and backward of two projections in a row, against differences in 64 bits."""
    N, K, r, L = 264, 328, 8, 3
    one, two = lora_inputs(M, N, K, r, L, 160), lora_inputs(M, K, N, r, L, 170)
    ids, target = ids_of("runs", M, L, 161), normal((M, K), 162)

    def forward(t, x, u=None):
        return tmg.lora_linear(x, t["W"], t["A"], t["B"], ids, scales=t["scales"], u=u)

    u1, u2 = torch.empty(M, r, dtype=BF16, device=DEV), torch.empty(M, r, dtype=BF16, device=DEV)
    h = forward(one, one["x"], u1)
    y = forward(two, h, u2)
    dy = (y.float() - target.float()).to(BF16)
    dh, dA2, dB2 = tmg.lora_linear_backward(dy, h, two["W"], two["A"], two["B"], ids, u2, scales=two["scales"])
    dx, dA1, dB1 = tmg.lora_linear_backward(dh, one["x"], one["W"], one["A"], one["B"], ids, u1, scales=one["scales"])
    tmg.check()

    def loss(x, A1, B1, A2, B2):
        v = x
        for t, A, B in ((one, A1, B1), (two, A2, B2)):
            z = v @ t["W"].to(W).T
            for l in range(L):
                on = (ids == l).to(W)[:, None] * t["scales"][l].to(W)
                z = z + on * ((v @ A[l].T) @ B[l].T)
            v = z
        return 0.5 * ((v - target.to(W)) ** 2).sum()

    at = [v.to(W) for v in (one["x"], one["A"], one["B"], two["A"], two["B"])]
    for i, g in enumerate((dx, dA1, dB1, dA2, dB2)):
        way = normal(at[i].shape, 180 + i).to(W)
        step = 1e-4
        there = [[v + sign * step * way if j == i else v for j, v in enumerate(at)] for sign in (1, -1)]
        slope = (loss(*there[0]) - loss(*there[1])) / (2 * step)
        # every entry of the gradient passes at most eight roundings to bf16, each of a random sign:
        # over the sum the relative error of its root of squares is below 8 * 2^-8
        bound = 8 * ROUND * (g.to(W) * way).pow(2).sum().sqrt() * 4 + 8 * ROUND * slope.abs()
        assert ((g.to(W) * way).sum() - slope).abs() <= bound, i


def test_lora_results_past_2_31_elements(tmg):
    """More than 2^31 elements of D and of dx; rows at both ends and around the border."""
    M, N, K, r, L = 66000, 33000, 64, 8, 3
    t = lora_inputs(M, N, K, r, L, 190)
    ids = ids_of("runs", M, L, 191)
    D = tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], ids, scales=t["scales"])
    tmg.check()
    rows = torch.tensor([0, 1, 130, 65075, 65076, 65077, M - 2, M - 1], device=DEV)
    want, err, _, _ = adapted(t["x"][rows], t["W"], t["A"], t["B"], ids[rows], t["scales"])
    close(D[rows], want, err)
    del D
    dD, u = normal((M, K), 192), normal((M, r), 193)
    b = lora_inputs(8, K, N, r, L, 194)
    x = torch.zeros(M, N, dtype=BF16, device=DEV)
    dx, dA, dB = tmg.lora_linear_backward(dD, x, b["W"], b["A"], b["B"], ids, u)
    tmg.check()
    (want, err), _, _ = gradients(dD[rows], x[rows], b["W"], b["A"], b["B"], ids[rows], u[rows])
    close(dx[rows], want, err)
    assert not dA.any()
    _, _, (want, err) = gradients(dD, x[:, :1], b["W"][:, :1], b["A"][:, :, :1], b["B"], ids, u)
    close(dB, want, err)
