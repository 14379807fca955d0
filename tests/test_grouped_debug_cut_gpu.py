"""Tiles cut over several CTA pairs through the bounds-checked build: every access to
their partial sums and counters checked, results equal to the normal build's."""
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def calls(t):
    g = torch.Generator().manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()
    out = [t.linear(rand(1000, 4096), rand(5120, 4096), activation="silu")]            # 24 tiles over three pairs each
    off = torch.tensor([0, 700, 1030], dtype=torch.int32).cuda()
    x, W = rand(1030, 4096), rand(2, 5120, 4096)
    out += [t.grouped_gemm(x, W, off), t.grouped_gemm(x, W, off, activation="swiglu")]
    deep, wide = rand(5000, 520), rand(5000, 300)
    for sizes in ([5000], [3100, 0, 1900]):
        o = torch.tensor([0] + sizes).cumsum(0).to(torch.int32).cuda()
        out.append(t.grouped_gemm_wgrad(wide, deep, o))
    dD, A, B = rand(2560, 2048), rand(2560, 2560), rand(2048, 2560)
    out += list(t.linear_backward(dD, A, B, preact=dD, activation="gelu"))             # the GEMM's stream-K tiles
    t.check()
    return [o.clone() for o in out]


def test_debug_build_checks_cut_tiles():
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
