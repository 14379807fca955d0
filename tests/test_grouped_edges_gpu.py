"""Edges of the grouped and dense products and their gradients: empty operands,
NaN and infinities through the activations, extents near the limits.  Inputs
are integers or powers of two, so results are exact."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def tmg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as t
    yield t
    t.check()


def ints(shape, seed):
    return torch.randint(-2, 3, shape, generator=torch.Generator().manual_seed(seed)).float().to(BF16)


def test_wgrad_without_rows_is_zero_whatever_the_workspace_holds(tmg):
    """R = 0 with row numbers given (an empty torch tensor has no address, so
    through the C ABI), after a call that gathered NaN."""
    from tiled_mma_atom_gb300 import _native
    N, K, E, T = 40, 64, 3, 50
    A, rows = torch.full((T, K), math.nan, dtype=BF16, device=DEV), torch.zeros(100, dtype=torch.int32, device=DEV)
    tmg.grouped_gemm_wgrad(torch.zeros(100, N, dtype=BF16, device=DEV), A,
                           torch.tensor([0, 30, 60, 100], dtype=torch.int32, device=DEV), rows=rows)
    dB = torch.full((E, N, K), 7.0, dtype=BF16, device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    d = torch.zeros(8, N, dtype=BF16, device=DEV)
    st = _native.lib().tmg_grouped_gemm_wgrad(d.data_ptr(), N, 1, A.data_ptr(), K, 1, dB.data_ptr(), off.data_ptr(),
                                              rows.data_ptr(), 0, N, K, E, T, torch.cuda.current_stream().cuda_stream)
    assert st == _native.OK
    tmg.check()
    assert (dB == 0).all()


@pytest.mark.parametrize("R", [5, 300, 4000])
@pytest.mark.parametrize("gather", [False, True])
def test_no_group_has_rows(tmg, R, gather):
    """What the routing leaves when every token is masked: rows, and none in a group."""
    N, K, E = 264, 136, 6
    A, B, d = ints((R, K), 12).to(DEV), ints((E, N, K), 13).to(DEV), ints((R, N), 14).to(DEV)
    r = tmg.moe_route(torch.full((R, E), -math.inf, device=DEV), 1)
    assert not r.offsets.any() and (r.rows == -1).all() and (r.slots == -1).all()
    rows = r.rows if gather else None
    for act, cols, pre in (("none", N, None), ("swiglu", N // 2, None), ("swiglu_grad", 2 * N, torch.ones(R, 2 * N, dtype=BF16, device=DEV))):
        D = torch.full((R, cols), 7.5, dtype=BF16, device=DEV)
        tmg.grouped_gemm(A, B, r.offsets, D, rows=rows, activation=act, preact=pre)
        assert (D == 7.5).all()
    assert not tmg.grouped_gemm_wgrad(d, A, r.offsets, rows=rows).any()
    out = tmg.moe_combine(A, r.slots, r.weights, residual=A)
    assert torch.equal(out, A)
    tmg.check()


@pytest.mark.parametrize("M,N,K", [(4, 264, 64), (900, 1000, 200), (5, 24, 0)])
def test_linear_relu_keeps_nan(tmg, M, N, K):
    """relu(NaN) is NaN, of -inf 0, of +inf +inf, in every kernel of the product."""
    A, B, bias = ints((M, K), 1), ints((N, K), 2), torch.zeros(N)
    bias[5], bias[6], bias[7] = math.nan, math.inf, -math.inf
    pre = torch.empty(M, N, dtype=BF16, device=DEV)
    D = tmg.linear(A.to(DEV), B.to(DEV), bias=bias.to(DEV), activation="relu", preact=pre)
    tmg.check()
    z = A.double() @ B.double().T + bias.double()
    want = torch.relu(z).to(BF16)
    assert torch.isnan(want[:, 5]).all()
    for got, ref in ((pre, z.to(BF16)), (D, want)):
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(ref))
        assert torch.equal(got.cpu().nan_to_num(1.0), ref.nan_to_num(1.0))


def test_linear_backward_of_very_wide_outputs(tmg):
    """More column blocks of dz than a grid has in its second dimension."""
    M, N, K = 3, 256 * 65535 + 8, 8
    A, B, pre = ints((M, K), 3).to(DEV), torch.zeros(N, K, dtype=BF16, device=DEV), torch.zeros(M, N, dtype=BF16, device=DEV)
    dD = torch.zeros(M, N, dtype=BF16, device=DEV)
    at = torch.tensor([0, 1000, 256 * 65535 - 1, 256 * 65535, N - 1], device=DEV)
    dD[:, at], pre[:, at], B[at] = ints((M, 5), 4).to(DEV), 1.0, ints((5, K), 5).to(DEV)
    pre[1, at[2]] = -1.0
    dA, dB, db = tmg.linear_backward(dD, A, B, preact=pre, activation="relu")
    tmg.check()
    dz = dD[:, at].double() * (pre[:, at] > 0)
    assert torch.equal(dA, (dz @ B[at].double()).to(BF16))
    assert torch.equal(dB[at], (dz.T @ A.double()).to(BF16)) and torch.equal(db[at].double(), dz.sum(0))
    dB[at], db[at] = 0, 0
    assert not dB.any() and not db.any()


TOP = 2 ** 31 - 8


@pytest.fixture
def patient(tmg):
    """Contractions of 2^31 terms take a second or so of one cluster: longer waits."""
    tmg.set_wait_budget_ns(60_000_000_000)
    yield tmg
    tmg.set_wait_budget_ns(2_000_000_000)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,N", [(1, 8), (3, 16)])
def test_linear_contraction_just_below_2_31(patient, M, N):
    A, B = torch.zeros(M, TOP, dtype=BF16, device=DEV), torch.zeros(N, TOP, dtype=BF16, device=DEV)
    at = torch.tensor([0, 77, 2 ** 30, TOP - 60, TOP - 1], device=DEV)
    A[:, at], B[:, at] = ints((M, 5), 6).to(DEV), ints((N, 5), 7).to(DEV)
    D = patient.linear(A, B)
    patient.check()
    assert torch.equal(D, (A[:, at].double() @ B[:, at].double().T).to(BF16))


def test_linear_columns_just_below_2_31(patient):
    K = 8
    A, B = ints((2, K), 8).to(DEV), torch.zeros(TOP, K, dtype=BF16, device=DEV)
    at = torch.tensor([0, 300, 2 ** 30, TOP - 9, TOP - 1], device=DEV)
    B[at] = ints((5, K), 9).to(DEV)
    D = patient.linear(A, B)
    patient.check()
    assert torch.equal(D[:, at], (A.double() @ B[at].double().T).to(BF16))
    D[:, at] = 0
    assert not D[0].any() and not D[1].any()


@pytest.mark.parametrize("sizes", [[0, TOP], [TOP - 40, 40]])
def test_grouped_rows_just_below_2_31(patient, sizes):
    N, K = 8, 8
    off = torch.tensor([0, sizes[0], TOP], dtype=torch.int32, device=DEV)
    A, B = torch.zeros(TOP, K, dtype=BF16, device=DEV), ints((2, N, K), 10).to(DEV)
    at = torch.tensor([0, 255, 2 ** 30, TOP - 41, TOP - 40, TOP - 1], device=DEV)
    A[at] = ints((6, K), 11).to(DEV)
    D = patient.grouped_gemm(A, B, off)
    dB = patient.grouped_gemm_wgrad(D, A, off)
    patient.check()
    want, grad = torch.zeros(6, N, device=DEV, dtype=torch.float64), torch.zeros(2, N, K, device=DEV, dtype=torch.float64)
    for i, r in enumerate(at.tolist()):
        e = 0 if r < sizes[0] else 1
        want[i] = B[e].double() @ A[r].double()
        grad[e] += torch.outer(want[i], A[r].double())
    assert torch.equal(D[at].double(), want) and torch.equal(dB, grad.to(BF16))
    D[at] = 0
    assert all(not part.any() for part in D.view(torch.int64).split(1 << 28))
