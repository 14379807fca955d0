"""GPU parity of the expert-grouped products (tmg_grouped_gemm and its weight
gradient) and of the dense product with bias, activation and residual
(tmg_linear and its gradient) against plain 64-bit evaluations on the CPU.

Bounds, from the arithmetic:
  * integer-valued inputs (|a|, |b| <= 2, K <= 4096): every fp32 sum is exact, so
    a result without activation is the bf16 rounding of the exact value, bit for
    bit;
  * otherwise a product z of K terms with S = sum |a b| is off by at most
    e = K 2^-22 S (fp32 sums in any order, with slack for the tensor core's
    alignment of addends), scales and bias add 2^-22 of their result; an
    activation of slope <= L passes L e on and adds 2^-16 of its scale (fast
    exponential and division); one bf16 rounding (8 significant bits) adds 2^-8 |y|.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
W = torch.float64


@pytest.fixture(scope="module")
def tmg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as t
    yield t
    t.check()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def ints(shape, seed, dtype=BF16):
    return torch.randint(-2, 3, shape, generator=gen(seed)).to(torch.float32).to(dtype)


def normal(shape, seed, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=gen(seed)) * std).to(dtype)


def offsets_of(sizes, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(sizes)]), dtype=torch.int32)


def groups(offsets):
    o = offsets.tolist()
    return [(e, slice(o[e], o[e + 1])) for e in range(len(o) - 1)]


def gathered(A, rows, R):
    """A's rows as the product reads them (64 bits): zeros where `rows` is out of range."""
    if rows is None:
        return A.to(W)
    ok = (rows >= 0) & (rows < A.shape[0])
    return A.to(W)[rows.long().clamp(0, max(A.shape[0] - 1, 0))] * ok[:, None]


def product(A, B, offsets, rows=None, scale_a=None, scale_b=None, R=None):
    """z and the error bound e of every row in a group, in 64 bits (NaN elsewhere)."""
    R = (A.shape[0] if rows is None else rows.shape[0]) if R is None else R
    a = gathered(A, rows, R)
    sa = None if scale_a is None else gathered(scale_a[:, None], rows, R)
    z = torch.full((R, B.shape[1]), math.nan, dtype=W)
    err = torch.zeros_like(z)
    for e, r in groups(offsets):
        b = B[e].to(W)
        z[r] = a[r] @ b.T
        err[r] = A.shape[1] * 2.0 ** -22 * (a[r].abs() @ b.abs().T)
        f = torch.ones(b.shape[0], dtype=W) if scale_b is None else scale_b[e].to(W)
        f = f * (1.0 if sa is None else sa[r])
        z[r] = z[r] * f
        err[r] = err[r] * f.abs() + 2.0 ** -22 * z[r].abs()
    return z, err


def silu(x):
    return x * torch.sigmoid(x)


def silu_slope(x):
    p = torch.sigmoid(x)
    return p * (1 + x * (1 - p))


def close(got, want, err, scale=None):
    got, scale = got.cpu().to(W), want.abs() if scale is None else scale
    there = ~torch.isnan(want)
    bound = (err + 2.0 ** -16 * scale + 2.0 ** -8 * 1.01 * (want.abs() + err) + 1e-30)[there]
    off = (got - want).abs()[there]
    assert torch.isfinite(got[there]).all()
    worst = (off / bound).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"off by {worst:.3g} of the bound"


def exact(got, want):
    there = ~torch.isnan(want)
    got, want = got.cpu()[there], want[there].to(torch.float32).to(BF16)
    assert torch.equal(got, want), f"{(got != want).sum().item()} of {got.numel()} differ"


def untouched(D, offsets, mark):
    o = offsets.tolist()
    assert (D[:o[0]] == mark).all() and (D[o[-1]:] == mark).all()


SIZES = {"one": [1], "empty": [0, 0, 0], "ragged": [0, 1, 37, 0, 300, 64, 0], "large": [700, 5, 513, 33, 256, 0],
         "many": [(7 * i) % 5 for i in range(130)]}


# ------------------------------------------------------------- grouped product

@pytest.mark.parametrize("N,K", [(8, 8), (136, 72), (520, 200), (257, 1000), (24, 1001), (300, 64)])
@pytest.mark.parametrize("sizes", ["one", "empty", "ragged", "large", "many"])
def test_grouped_exact(tmg, sizes, N, K):
    off = offsets_of(SIZES[sizes])
    R, E = int(off[-1]), len(SIZES[sizes])
    A, B = ints((R, K), 1), ints((E, N, K), 2)
    D = tmg.grouped_gemm(A.to(DEV), B.to(DEV), off.to(DEV))
    tmg.check()
    exact(D, product(A, B, off)[0])


@pytest.mark.parametrize("K", [64, 136, 1003])
def test_grouped_gather_exact(tmg, K):
    """Rows repeated, in any order, and out of range (read as zeros)."""
    off = offsets_of(SIZES["ragged"])
    R, E, N, T = int(off[-1]), 7, 264, 90
    A, B = ints((T, K), 3), ints((E, N, K), 4)
    rows = torch.randint(0, T, (R,), generator=gen(5)).int()
    rows[3], rows[50], rows[60], rows[61] = -1, T, T - 1, 2 ** 31 - 1
    D = tmg.grouped_gemm(A.to(DEV), B.to(DEV), off.to(DEV), rows=rows.to(DEV))
    tmg.check()
    exact(D, product(A, B, off, rows)[0])


def test_grouped_rows_outside_groups_are_left(tmg):
    off = offsets_of([5, 0, 40], first=3)
    R, N, K = 60, 72, 64
    A, B = ints((R, K), 6), ints((3, N, K), 7)
    D = torch.full((R, N), 7.5, dtype=BF16, device=DEV)
    tmg.grouped_gemm(A.to(DEV), B.to(DEV), off.to(DEV), D)
    tmg.check()
    exact(D, product(A, B, off)[0])
    untouched(D, off, 7.5)


@pytest.mark.parametrize("K", [64, 200])
def test_grouped_transposed_weights_exact(tmg, K):
    """B given as (E, K, N) transposed: the gradient of A."""
    off = offsets_of(SIZES["large"])
    R, E, N = int(off[-1]), 6, 328
    A, Bt = ints((R, K), 8), ints((E, K, N), 9)
    D = tmg.grouped_gemm(A.to(DEV), Bt.to(DEV).transpose(1, 2), off.to(DEV))
    tmg.check()
    exact(D, product(A, Bt.transpose(1, 2), off)[0])


@pytest.mark.parametrize("pad", [(0, 8, 8), (1, 3, 5), (4, 4, 1)])
def test_grouped_strides_exact(tmg, pad):
    """Operands and result as slices of larger tensors, aligned or not."""
    pa, pb, pd = pad
    off = offsets_of(SIZES["ragged"])
    R, E, N, K = int(off[-1]), 7, 144, 128
    A, B = ints((R, K + 16), 10), ints((E, N + 3, K + 16), 11)
    D = torch.full((R, N + 16), 7.5, dtype=BF16, device=DEV)
    a, b = A[:, pa:pa + K], B[:, 2:2 + N, pb:pb + K]
    tmg.grouped_gemm(A.to(DEV)[:, pa:pa + K], B.to(DEV)[:, 2:2 + N, pb:pb + K], off.to(DEV), D[:, pd:pd + N])
    tmg.check()
    exact(D[:, pd:pd + N].contiguous(), product(a, b, off)[0])
    assert (D[:, :pd] == 7.5).all() and (D[:, pd + N:] == 7.5).all()


def test_grouped_broadcast_rows_and_weights(tmg):
    """Stride 0: one row for all, one expert's weights for all."""
    off = offsets_of([3, 70, 0, 10])
    A, B = ints((1, 72), 12), ints((1, 40, 72), 13)
    D = tmg.grouped_gemm(A.to(DEV).expand(83, 72), B.to(DEV).expand(4, 40, 72), off.to(DEV))
    tmg.check()
    exact(D, product(A.expand(83, 72), B.expand(4, 40, 72), off)[0])


def test_grouped_nan_and_infinity_stay_in_their_rows(tmg):
    off = offsets_of([20, 0, 45])
    A, B = ints((65, 64), 14), ints((3, 48, 64), 15)
    A[7, 3], A[30, 5] = math.nan, math.inf
    D = tmg.grouped_gemm(A.to(DEV), B.to(DEV), off.to(DEV)).cpu()
    tmg.check()
    keep = [i for i in range(65) if i not in (7, 30)]
    A[7], A[30] = 0, 0
    exact(D[keep], product(A, B, off)[0][keep])
    assert torch.isnan(D[7]).all() and not torch.isfinite(D[30].float()).all()


def test_grouped_offsets_beyond_the_rows_are_clamped(tmg):
    off = torch.tensor([-5, 20, 10, 500], dtype=torch.int32)     # falling, and past the end
    R, N, K = 48, 40, 64
    A, B = ints((R, K), 16), ints((3, N, K), 17)
    D = torch.full((R, N), 7.5, dtype=BF16, device=DEV)
    tmg.grouped_gemm(A.to(DEV), B.to(DEV), off.to(DEV), D)
    tmg.check()
    assert torch.equal(D.cpu()[:10], (A[:10].float() @ B[0].float().T).to(BF16))
    assert torch.equal(D.cpu()[20:], (A[20:].float() @ B[2].float().T).to(BF16))


def test_grouped_k0(tmg):
    off = offsets_of([3, 4])
    D = tmg.grouped_gemm(torch.empty(7, 0, dtype=BF16, device=DEV), torch.empty(2, 24, 0, dtype=BF16, device=DEV),
                         off.to(DEV))
    tmg.check()
    assert (D == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("sizes", ["ragged", "large"])
def test_grouped_scales(tmg, kind, sizes):
    off = offsets_of(SIZES[sizes])
    R, E, N, K, T = int(off[-1]), len(SIZES[sizes]), 272, 400, 77
    dt = BF16 if kind == "bf16" else E4M3
    A, B = normal((T, K), 18, dtype=dt), normal((E, N, K), 19, dtype=dt)
    rows = torch.randint(0, T, (R,), generator=gen(20)).int()
    sa, sb = torch.rand(T, generator=gen(21)) + 0.5, torch.rand(E, N, generator=gen(22)) + 0.5
    D = tmg.grouped_gemm(A.to(DEV), B.to(DEV), off.to(DEV), rows=rows.to(DEV), scale_a=sa.to(DEV), scale_b=sb.to(DEV))
    tmg.check()
    close(D, *product(A, B, off, rows, sa, sb))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("sizes", ["one", "ragged", "large"])
@pytest.mark.parametrize("F", [8, 136, 260, 45])
@pytest.mark.parametrize("save", [False, True])
def test_grouped_swiglu(tmg, kind, sizes, F, save):
    off = offsets_of(SIZES[sizes])
    R, E, K, T = int(off[-1]), len(SIZES[sizes]), 208, 50
    dt = BF16 if kind == "bf16" else E4M3
    A, B = normal((T, K), 23, dtype=dt), normal((E, 2 * F, K), 24, K ** -0.5 if kind == "bf16" else 1.0, dtype=dt)
    rows = torch.randint(0, T, (R,), generator=gen(25)).int()
    sa, sb = (None, None) if kind == "bf16" else (torch.rand(T, generator=gen(26)) * 0.1,
                                                  torch.rand(E, 2 * F, generator=gen(27)) + 0.5)
    up = lambda t: None if t is None else t.to(DEV)
    pre = torch.full((R, 2 * F), 7.5, dtype=BF16, device=DEV) if save else None
    D = tmg.grouped_gemm(A.to(DEV), B.to(DEV), off.to(DEV), rows=rows.to(DEV), activation="swiglu", preact=pre,
                         scale_a=up(sa), scale_b=up(sb))
    tmg.check()
    z, err = product(A, B, off, rows, sa, sb)
    g, u, eg, eu = z[:, :F], z[:, F:], err[:, :F], err[:, F:]
    close(D, silu(g) * u, 1.1 * eg * u.abs() + silu(g).abs() * eu + eg * eu, (g * u).abs())
    if save:
        close(pre, z, err)


@pytest.mark.parametrize("F", [8, 200, 45])
@pytest.mark.parametrize("sizes", ["ragged", "large"])
def test_grouped_swiglu_grad(tmg, F, sizes):
    off = offsets_of(SIZES[sizes])
    R, E, H = int(off[-1]), len(SIZES[sizes]), 176
    dY, W2 = normal((R, H), 28), normal((E, H, F), 29, F ** -0.5)
    pre = normal((R, 2 * F), 30, 2.0)
    D = tmg.grouped_gemm(dY.to(DEV), W2.to(DEV).transpose(1, 2), off.to(DEV), activation="swiglu_grad",
                         preact=pre.to(DEV))
    tmg.check()
    da, err = product(dY, W2.transpose(1, 2), off)
    g, u = pre[:, :F].to(W), pre[:, F:].to(W)
    slope = silu_slope(g)
    want = torch.cat([da * u * slope, da * silu(g)], 1)
    size = torch.cat([(da * u).abs() * (1 + g.abs()), (da * g).abs()], 1)
    close(D, want, torch.cat([err * (u * slope).abs(), err * silu(g).abs()], 1), size)
    # and against differences of the SwiGLU itself
    h = 1e-5
    dg = (silu(g + h) - silu(g - h)) / (2 * h) * u * da
    there = ~torch.isnan(da)
    assert torch.allclose(want[:, :F][there], dg[there], rtol=1e-6, atol=1e-8)


def test_grouped_deterministic(tmg):
    off = offsets_of(SIZES["large"]).to(DEV)
    A, B = normal((int(off[-1]), 1024), 31).to(DEV), normal((6, 512, 1024), 32).to(DEV)
    first = tmg.grouped_gemm(A, B, off)
    for _ in range(3):
        assert torch.equal(first, tmg.grouped_gemm(A, B, off))
    tmg.check()


@pytest.mark.parametrize("sizes", [[4], [1, 0, 2], [40], [130, 3]])
@pytest.mark.parametrize("N,K", [(512, 4096), (2048, 1024), (264, 2000)])
def test_grouped_few_rows_exact(tmg, sizes, N, K):
    """Few tiles for the SMs: contractions split between them.  Twice: their
    counters come back to zero."""
    off = offsets_of(sizes)
    A, B = ints((int(off[-1]), K), 33), ints((len(sizes), N, K), 34)
    dA, dB, dO = A.to(DEV), B.to(DEV), off.to(DEV)
    D1 = tmg.grouped_gemm(dA, dB, dO)
    D2 = tmg.grouped_gemm(dA, dB, dO)
    tmg.check()
    want = product(A, B, off)[0]
    exact(D1, want)
    exact(D2, want)


@pytest.mark.parametrize("sizes", [[700, 330], [0, 1000, 3, 0]])
@pytest.mark.parametrize("activation", ["none", "swiglu"])
def test_grouped_cut_tiles(tmg, sizes, activation):
    """A last wave of few tiles with a long contraction: cut over several CTA pairs."""
    off, N, K = offsets_of(sizes), 5120, 4096
    R = int(off[-1])
    A, B = normal((R, K), 93), normal((len(sizes), N, K), 94, K ** -0.5)
    dA, dB, dO = A.to(DEV), B.to(DEV), off.to(DEV)
    outs = [tmg.grouped_gemm(dA, dB, dO, activation=activation) for _ in range(3)]
    tmg.check()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    z, err = product(A, B, off)
    if activation == "none":
        close(outs[0], z, err)
    else:
        g, u, eg, eu = z[:, :N // 2], z[:, N // 2:], err[:, :N // 2], err[:, N // 2:]
        close(outs[0], silu(g) * u, 1.1 * eg * u.abs() + silu(g).abs() * eu + eg * eu, (g * u).abs())


def test_grouped_one_group_takes_all(tmg):
    """All rows in one of many groups: more row tiles than an even spread has."""
    sizes = [0] * 20 + [3000] + [0] * 11
    off = offsets_of(sizes)
    A, B = ints((3000, 96), 35), ints((32, 136, 96), 36)
    D = tmg.grouped_gemm(A.to(DEV), B.to(DEV), off.to(DEV))
    tmg.check()
    exact(D, product(A, B, off)[0])


def test_grouped_offsets_past_32_bits(tmg):
    """Elements of B beyond 2^31."""
    E, N, K = 260, 2048, 4224
    B = torch.zeros((E, N, K), dtype=BF16, device=DEV)
    last = ints((N, K), 37)
    B[E - 1] = last.to(DEV)
    sizes = [0] * (E - 1) + [9]
    A = ints((9, K), 38)
    D = tmg.grouped_gemm(A.to(DEV), B, offsets_of(sizes).to(DEV))
    tmg.check()
    exact(D, A.to(W) @ last.to(W).T)


def test_grouped_on_another_stream(tmg):
    off = offsets_of(SIZES["large"])
    A, B = ints((int(off[-1]), 256), 39), ints((6, 264, 256), 40)
    dA, dB, dO = A.to(DEV), B.to(DEV), off.to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    D = tmg.grouped_gemm(dA, dB, dO, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    exact(D, product(A, B, off)[0])
    tmg.check(s)


def test_captured_graph_survives_growing_workspace(tmg):
    """A graph with a split contraction (partials in workspace), replayed after
    larger calls on the same stream have outgrown its workspace."""
    A, B, off = ints((4, 4096), 53), ints((1, 512, 4096), 54), offsets_of([4])
    dA, dB, dO, D = A.to(DEV), B.to(DEV), off.to(DEV), torch.empty((4, 512), dtype=BF16, device=DEV)
    big, W, o2 = ints((900, 4096), 55).to(DEV), ints((2, 520, 4096), 56).to(DEV), offsets_of([300, 600]).to(DEV)
    rows = torch.arange(900, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tmg.grouped_gemm(dA, dB, dO, D)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            tmg.grouped_gemm(dA, dB, dO, D)
        tmg.grouped_gemm(big, W, o2, rows=rows)
        tmg.grouped_gemm_wgrad(big, big, o2)
        D.zero_()
        for _ in range(2):
            g.replay()
    torch.cuda.current_stream().wait_stream(s)
    exact(D, product(A, B, off)[0])
    tmg.check(s)


# ------------------------------------------------------------- weight gradient

def wgrad(dD, A, off, rows):
    a = gathered(A, rows, dD.shape[0])
    d = dD.to(W)
    return torch.stack([d[r].T @ a[r] for _, r in groups(off)])


@pytest.mark.parametrize("N,K", [(8, 8), (264, 136), (512, 72), (45, 300)])
@pytest.mark.parametrize("sizes", ["one", "empty", "ragged", "large", "many"])
@pytest.mark.parametrize("gather", [False, True])
def test_wgrad_exact(tmg, sizes, N, K, gather):
    off = offsets_of(SIZES[sizes])
    R, T = int(off[-1]), 60
    dD, A = ints((R, N), 41), ints((T if gather else R, K), 42)
    rows = torch.randint(-1, T + 1, (R,), generator=gen(43)).int() if gather else None
    dB = tmg.grouped_gemm_wgrad(dD.to(DEV), A.to(DEV), off.to(DEV), rows=rows.to(DEV) if gather else None)
    tmg.check()
    exact(dB, wgrad(dD, A, off, rows))


@pytest.mark.parametrize("sizes", [[3, 18, 33, 0, 71], [130, 64, 1]])
def test_wgrad_groups_do_not_leak(tmg, sizes):
    """NaN and infinities in one group's rows (either operand) stay out of its
    neighbours, wherever the group ends inside a tile."""
    off = offsets_of(sizes)
    R, N, K = int(off[-1]), 264, 136
    dD, A = ints((R, N), 44), ints((R, K), 45)
    want = wgrad(dD, A, off, None)
    bad = 1
    dD[off[bad], :], A[off[bad + 1] - 1, :] = math.nan, math.inf
    dB = tmg.grouped_gemm_wgrad(dD.to(DEV), A.to(DEV), off.to(DEV)).cpu()
    tmg.check()
    keep = [e for e in range(len(sizes)) if e != bad]
    exact(dB[keep], want[keep])
    assert not torch.isfinite(dB[bad].float()).any()


@pytest.mark.parametrize("sizes", [[2500], [900, 30]])
def test_wgrad_split_contraction_exact(tmg, sizes):
    """Few output tiles, a long contraction."""
    off = offsets_of(sizes)
    R, N, K = int(off[-1]), 256, 200
    dD, A = ints((R, N), 46), ints((R, K), 47)
    dB1 = tmg.grouped_gemm_wgrad(dD.to(DEV), A.to(DEV), off.to(DEV))
    dB2 = tmg.grouped_gemm_wgrad(dD.to(DEV), A.to(DEV), off.to(DEV))
    tmg.check()
    exact(dB1, wgrad(dD, A, off, None))
    assert torch.equal(dB1, dB2)


@pytest.mark.parametrize("sizes", [[3000], [5000, 3000], [4100, 0, 3900]])
def test_wgrad_few_tiles_of_many_rows_exact(tmg, sizes):
    """Tiles cut over several CTA pairs, in one group and across groups."""
    off, N, K = offsets_of(sizes), 300, 520
    R = int(off[-1])
    d, A = ints((R, N), 91), ints((R, K), 92)
    first = None
    for _ in range(3):
        dB = tmg.grouped_gemm_wgrad(d.to(DEV), A.to(DEV), off.to(DEV))
        tmg.check()
        first = dB if first is None else first
        assert torch.equal(dB, first)
    exact(first, torch.stack([d[r].to(W).T @ A[r].to(W) for _, r in groups(off)]))


def test_wgrad_strides(tmg):
    off = offsets_of(SIZES["ragged"])
    R, N, K = int(off[-1]), 72, 80
    dD, A = ints((R, N + 9), 48), ints((K, R), 49)
    dB = tmg.grouped_gemm_wgrad(dD.to(DEV)[:, 3:3 + N], A.to(DEV).T, off.to(DEV))
    tmg.check()
    exact(dB, wgrad(dD[:, 3:3 + N], A.T, off, None))


def test_gradients_against_differences(tmg):
    """The input and weight gradients against central differences of the
    64-bit product along random directions."""
    off = offsets_of([5, 0, 33])
    R, N, K = 38, 40, 64
    A, B, dD = normal((R, K), 50), normal((3, N, K), 51), normal((R, N), 52)
    dA = tmg.grouped_gemm(dD.to(DEV), B.to(DEV).transpose(1, 2), off.to(DEV)).cpu().to(W)
    dB = tmg.grouped_gemm_wgrad(dD.to(DEV), A.to(DEV), off.to(DEV)).cpu().to(W)
    tmg.check()
    loss = lambda a, b: sum(((a[r] @ b[e].T) * dD[r].to(W)).sum() for e, r in groups(off))
    a, b, h = A.to(W), B.to(W), 1e-3
    for seed in range(4):
        va, vb = torch.randn(R, K, dtype=W, generator=gen(seed)), torch.randn(3, N, K, dtype=W, generator=gen(seed + 9))
        # a gradient entry is off by at most 2^-8 of itself; a random direction adds the entries' errors in quadrature
        for grad, v, diff in ((dA, va, loss(a + h * va, b) - loss(a - h * va, b)),
                              (dB, vb, loss(a, b + h * vb) - loss(a, b - h * vb))):
            assert abs((grad * v).sum() - diff / (2 * h)) <= 6 * 2.0 ** -9 * (grad * v).norm()


# --------------------------------------------------------------- dense product

ACTS = {"none": (lambda z: z, 1.0, lambda z: torch.ones_like(z)),
        "relu": (lambda z: z.clamp(min=0), 1.0, lambda z: (z > 0).to(z.dtype)),
        "silu": (silu, 1.1, silu_slope),
        "gelu": (lambda z: 0.5 * z * torch.erfc(-z / math.sqrt(2)), 1.13,
                 lambda z: 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))}


@pytest.mark.parametrize("M", [1, 3, 16, 33, 130, 300, 1025])
@pytest.mark.parametrize("N,K", [(8, 8), (264, 136), (1000, 520), (45, 77)])
def test_linear_exact(tmg, M, N, K):
    """No activation: bias and residual are integers too."""
    A, B, res = ints((M, K), 60), ints((N, K), 61), ints((M, N), 62)
    bias = torch.randint(-8, 9, (N,), generator=gen(63)).float()
    D = tmg.linear(A.to(DEV), B.to(DEV), bias=bias.to(DEV), residual=res.to(DEV))
    tmg.check()
    exact(D, A.to(W) @ B.to(W).T + bias.to(W) + res.to(W))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("M", [2, 70, 513])
def test_linear_epilogue(tmg, kind, act, M):
    N, K = 264, 400
    dt = BF16 if kind == "bf16" else E4M3
    A, B, res = normal((M, K), 64, dtype=dt), normal((N, K), 65, dtype=dt), normal((M, N), 66)
    sa, sb = torch.rand(M, generator=gen(67)) * 0.2, torch.rand(N, generator=gen(68)) + 0.2
    bias = torch.randn(N, generator=gen(69))
    pre = torch.empty((M, N), dtype=BF16, device=DEV)
    D = tmg.linear(A.to(DEV), B.to(DEV), bias=bias.to(DEV), activation=act, residual=res.to(DEV), preact=pre,
                   scale_a=sa.to(DEV), scale_b=sb.to(DEV))
    tmg.check()
    z, err = product(A, B[None], offsets_of([M]), None, sa, sb[None])
    z = z + bias.to(W)
    err = err + 2.0 ** -22 * (z.abs() + bias.to(W).abs())
    f, slope, _ = ACTS[act]
    close(pre, z, err)
    y = f(z) + res.to(W)
    close(D, y, slope * err + 2.0 ** -22 * y.abs(), z.abs())


def test_linear_residual_in_place_and_strides(tmg):
    M, N, K = 150, 200, 96
    A, B, X = ints((M, K), 70), ints((N, K), 71), ints((M, N + 24), 72)
    dX = X.to(DEV)
    out = tmg.linear(A.to(DEV), B.to(DEV), dX[:, 8:8 + N], residual=dX[:, 8:8 + N])
    tmg.check()
    exact(out.contiguous(), A.to(W) @ B.to(W).T + X[:, 8:8 + N].to(W))
    assert torch.equal(dX[:, :8].cpu(), X[:, :8]) and torch.equal(dX[:, 8 + N:].cpu(), X[:, 8 + N:])


def test_linear_transposed_operands_exact(tmg):
    M, N, K = 260, 136, 72
    A, B = ints((K, M), 73), ints((K, N), 74)
    D = tmg.linear(A.to(DEV).T, B.to(DEV).T)
    tmg.check()
    exact(D, A.T.to(W) @ B.to(W))


def test_linear_k0_is_the_epilogue(tmg):
    bias, res = torch.randn(24, generator=gen(75)), normal((5, 24), 76)
    D = tmg.linear(torch.empty(5, 0, dtype=BF16, device=DEV), torch.empty(24, 0, dtype=BF16, device=DEV),
                   bias=bias.to(DEV), activation="silu", residual=res.to(DEV))
    tmg.check()
    z = bias.to(W).expand(5, 24)
    close(D, silu(z) + res.to(W), torch.zeros_like(z), z.abs())


@pytest.mark.parametrize("M,N,K", [(4, 4096, 4096), (16, 1000, 8192), (1, 8192, 1024), (200, 512, 4000)])
def test_linear_few_rows_exact(tmg, M, N, K):
    A, B = ints((M, K), 77), ints((N, K), 78)
    bias = torch.randint(-8, 9, (N,), generator=gen(79)).float()
    res = ints((M, N), 80)
    want = A.to(W) @ B.to(W).T + bias.to(W) + res.to(W)
    for _ in range(2):
        D = tmg.linear(A.to(DEV), B.to(DEV), bias=bias.to(DEV), residual=res.to(DEV))
        tmg.check()
        exact(D, want)


@pytest.mark.parametrize("M,N,K", [(1000, 5120, 4096), (300, 10000, 4000), (2000, 2700, 4100)])
def test_linear_cut_tiles_exact(tmg, M, N, K):
    """A last wave of few tiles with a long contraction, with everything the epilogue takes."""
    A, B, res = ints((M, K), 95), ints((N, K), 96), ints((M, N), 97)
    bias = torch.randint(-8, 9, (N,), generator=gen(98)).float()
    pre = torch.zeros((M, N), dtype=BF16, device=DEV)
    z = (A.to(DEV).double() @ B.to(DEV).double().T).cpu() + bias.to(W)
    for _ in range(2):
        D = tmg.linear(A.to(DEV), B.to(DEV), bias=bias.to(DEV), activation="relu", residual=res.to(DEV), preact=pre)
        tmg.check()
        exact(pre, z)
        exact(D, z.clamp(min=0) + res.to(W))


@pytest.mark.parametrize("M,N,K", [(16, 1000, 2048), (150, 1000, 96), (900, 1000, 200), (2500, 1000, 64)])
def test_linear_residual_in_place_exact(tmg, M, N, K):
    A, B, X = ints((M, K), 81), ints((N, K), 82), ints((M, N), 83)
    dX = X.to(DEV)
    tmg.linear(A.to(DEV), B.to(DEV), dX, residual=dX)
    tmg.check()
    exact(dX, A.to(W) @ B.to(W).T + X.to(W))


@pytest.mark.parametrize("M", [1, 40, 700])
def test_calls_in_a_row_see_each_other(tmg, M):
    """Launches overlap: every call reads what the one before wrote, as its rows, its
    residual and (a signed permutation, made by a product itself) its weight."""
    K, steps = 512, 6
    perm = torch.randperm(K, generator=gen(84))
    sign = (torch.randint(0, 2, (K,), generator=gen(85)) * 2 - 1).float()
    P = torch.zeros(K, K)
    P[torch.arange(K), perm] = sign
    x0 = torch.randint(-1, 2, (M, K), generator=gen(86)).float()
    want = [x0]
    for _ in range(steps):
        want.append(want[-1] @ P.T + want[-1])
    dP, eye, x, zero = (t.to(BF16).to(DEV) for t in (P, torch.eye(K), x0, torch.zeros(K, K)))
    for _ in range(20):
        y, w = x, zero.clone()
        for i in range(steps):
            tmg.linear(eye, dP.T.contiguous(), w)         # w = P again
            y = tmg.linear(y, w, residual=y)
            w.zero_() if i % 2 else tmg.linear(eye, zero, w)
        g = tmg.grouped_gemm(y, dP[None], torch.tensor([0, M], dtype=torch.int32, device=DEV))
        assert torch.equal(y.cpu().float(), want[-1])
        assert torch.equal(g.cpu().float(), want[-1] @ P.T)
    tmg.check()


def test_linear_results_past_32_bits(tmg):
    """More than 2^31 elements of D, of the residual and of preact."""
    M, N, K = 280000, 8192, 16
    A, B = ints((M, K), 87).to(DEV), ints((N, K), 88).to(DEV)
    res = torch.ones((M, N), dtype=BF16, device=DEV)
    pre = torch.empty_like(res)
    D = tmg.linear(A, B, residual=res, preact=pre)
    tmg.check()
    for r in (slice(0, 50), slice(M - 50, M)):
        z = A[r].cpu().to(W) @ B.cpu().to(W).T
        exact(pre[r], z)
        exact(D[r], z + 1)


def test_wgrad_results_past_32_bits(tmg):
    E, N, K, R = 260, 2048, 4224, 40
    off = offsets_of([0] * (E - 1) + [R])
    d, A = ints((R, N), 89), ints((R, K), 90)
    dB = tmg.grouped_gemm_wgrad(d.to(DEV), A.to(DEV), off.to(DEV))
    tmg.check()
    exact(dB[E - 1], d.to(W).T @ A.to(W))
    assert not dB[E - 2].any() and not dB[0].any()


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (77, 136, 64), (600, 264, 200), (130, 45, 33), (0, 16, 8)])
def test_linear_backward(tmg, act, M, N, K):
    A, B, dD, pre = normal((M, K), 81), normal((N, K), 82), normal((M, N), 83), normal((M, N), 84, 2.0)
    dA, dB, db = tmg.linear_backward(dD.to(DEV), A.to(DEV), B.to(DEV), preact=pre.to(DEV), activation=act)
    tmg.check()
    f, _, slope = ACTS[act]
    z = pre.to(W)
    dz = dD.to(W) * slope(z)
    h = 1e-5
    diff = (f(z + h) - f(z - h)) / (2 * h) * dD.to(W)
    smooth = z.abs() > 2 * h
    assert torch.allclose(dz[smooth], diff[smooth], rtol=1e-6, atol=1e-8)
    # dz enters the products rounded to bf16 (not for "none"), and with the fast functions' error
    edz = dD.to(W).abs() * (1 + z.abs()) * 2.0 ** -16 + (0 if act == "none" else 2.0 ** -8) * dz.abs()
    close(dA, dz @ B.to(W), edz @ B.to(W).abs() + N * 2.0 ** -22 * (dz.abs() @ B.to(W).abs()))
    close(dB, dz.T @ A.to(W), edz.T @ A.to(W).abs() + M * 2.0 ** -22 * (dz.T.abs() @ A.to(W).abs()))
    eb = (dD.to(W).abs() * (1 + z.abs())).sum(0) * 2.0 ** -16 + M * 2.0 ** -23 * dz.abs().sum(0) + 1e-30
    assert ((db.cpu().to(W) - dz.sum(0)).abs() <= eb).all()


# -------------------------------------------------------------------- refusals

def test_refusals(tmg):
    A, B = torch.zeros(8, 64, dtype=BF16, device=DEV), torch.zeros(2, 16, 64, dtype=BF16, device=DEV)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    for call in (lambda: tmg.grouped_gemm(A, B, off.long()), lambda: tmg.grouped_gemm(A, B, off[:2]),
                 lambda: tmg.grouped_gemm(A, B[:, :, :32], off), lambda: tmg.grouped_gemm(A, B, off, activation="gelu"),
                 lambda: tmg.grouped_gemm(A, B, off, activation="swiglu_grad"),
                 lambda: tmg.grouped_gemm(A, B, off, rows=off.float()),
                 lambda: tmg.grouped_gemm(A, B, off, preact=A), lambda: tmg.grouped_gemm(A.cpu(), B, off),
                 lambda: tmg.grouped_gemm_wgrad(A, A[:4], off), lambda: tmg.linear(A, B[0][:, :32]),
                 lambda: tmg.linear(A, B[0], activation="swiglu"), lambda: tmg.linear(A, B[0], residual=A),
                 lambda: tmg.linear_backward(A, A, B[0]), lambda: tmg.linear(A, B[0], bias=torch.zeros(16, device=DEV).half()),
                 lambda: tmg.linear_backward(torch.zeros(8, 16, dtype=BF16, device=DEV), A, B[0], activation="gelu")):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        tmg.grouped_gemm(A.float(), B.float(), off)
    with pytest.raises(TypeError):
        tmg.linear(A, B[0].to(E4M3))
    with pytest.raises(tmg.TmgError):
        tmg.grouped_gemm(A, torch.zeros(2, 15, 64, dtype=BF16, device=DEV), off, activation="swiglu",
                         D=torch.zeros(8, 7, dtype=BF16, device=DEV))
