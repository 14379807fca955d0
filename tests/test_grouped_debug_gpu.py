"""The grouped and dense products, their gradients and the routing through the
bounds-checked build (libtmg_debug.so): every store and every access to split
partials checked, results equal to the normal build's bit for bit."""
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def calls(t):
    g = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()
    out = []
    for sizes, N, K in (([0, 1, 37, 300, 64], 136, 200), ([3, 1], 512, 4096), ([700, 20], 264, 72)):
        E, R = len(sizes), sum(sizes)
        off = torch.tensor([0] + sizes).cumsum(0).to(torch.int32).cuda()
        x, W, rows = rand(50, K), rand(E, N, K), torch.randint(0, 50, (R,), generator=g).int().cuda()
        d, pre = rand(R, N), rand(R, 2 * K)
        saved = torch.empty(R, N, dtype=BF16, device="cuda")
        out += [t.grouped_gemm(x, W, off, rows=rows), t.grouped_gemm(x, W, off, rows=rows, activation="swiglu", preact=saved),
                saved, t.grouped_gemm(d, W.transpose(1, 2), off, activation="swiglu_grad", preact=pre),
                t.grouped_gemm_wgrad(d, x, off, rows=rows)]
    for M, N, K in ((3, 512, 4096), (300, 264, 136), (70, 45, 77)):
        A, B, res, bias = rand(M, K), rand(N, K), rand(M, N), torch.randn(N, generator=g).cuda()
        pre = torch.empty(M, N, dtype=BF16, device="cuda")
        out += [t.linear(A, B, bias=bias, activation="gelu", residual=res, preact=pre), pre]
        out += list(t.linear_backward(res, A, B, preact=pre, activation="gelu"))
    r = t.moe_route(rand(300, 40), 6)
    Y = rand(1800, 104)
    out += list(r) + [t.moe_combine(Y, r.slots, r.weights)] + list(t.moe_combine_backward(rand(300, 104), Y, r.slots, r.weights))
    t.check()
    return [o.clone() for o in out]


def test_debug_build_is_clean_and_equal():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as t
    from tiled_mma_atom_gb300 import _native, build
    build.build(debug_bounds=True)
    want = calls(t)
    _native.use_library(_native.DEBUG_LIB_PATH)
    try:
        assert _native.lib().tmg_debug_build() == 1
        got = calls(t)
    finally:
        _native.use_library(os.path.join(_native.HERE, "libtmg.so"))
    for a, b in zip(want, got):
        assert torch.equal(a, b)
