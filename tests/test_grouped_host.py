"""Host-side checks of the grouped products, the dense product with residual
and the routing (no GPU): what they refuse before any device work, and what
is empty."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def native():
    from tiled_mma_atom_gb300 import build
    build.build()
    from tiled_mma_atom_gb300 import _native
    return _native


def grouped(native, **over):
    v = dict(A=16, B=16, D=16, offsets=16, rows=None, scale_a=None, scale_b=None, preact=None, R=8, N=16, K=64, E=2, T=8,
             lda=64, a_col=1, b_expert=1024, b_row=64, b_col=1, ldd=32, ld_preact=32, in_dtype=native.BF16, activation=0)
    v.update(over)
    return native.lib().tmg_grouped_gemm(ctypes.byref(native.GroupedArgs(**v)), None)


def linear(native, **over):
    v = dict(A=16, B=16, D=16, scale_a=None, scale_b=None, bias=None, residual=None, preact=None, M=8, N=16, K=64, lda=64,
             a_col=1, b_row=64, b_col=1, ldd=16, ld_residual=0, ld_preact=0, in_dtype=native.BF16, activation=0)
    v.update(over)
    return native.lib().tmg_linear(ctypes.byref(native.LinearArgs(**v)), None)


def test_struct_layouts(native):
    assert ctypes.sizeof(native.GroupedArgs) == 8 * 8 + 12 * 8 + 8
    assert ctypes.sizeof(native.LinearArgs) == 8 * 8 + 10 * 8 + 8


@pytest.mark.parametrize("over", [dict(R=-1), dict(N=-1), dict(K=-1), dict(E=0), dict(E=1025), dict(activation=1),
                                  dict(activation=9), dict(in_dtype=7), dict(activation=4, N=15), dict(activation=5),
                                  dict(activation=5, preact=16, ld_preact=31), dict(ldd=15), dict(lda=-64),
                                  dict(b_expert=-1), dict(offsets=None), dict(D=None), dict(A=None), dict(B=None),
                                  dict(activation=4, preact=16, ld_preact=15), dict(b_expert=2 ** 61)])
def test_grouped_refuses(native, over):
    assert grouped(native, **over) == native.ERR_INVALID_ARG
    assert native.lib().tmg_last_error()


def test_grouped_unsupported_and_empty(native):
    assert grouped(native, in_dtype=native.F32) == native.ERR_UNSUPPORTED
    assert grouped(native, R=2 ** 31, T=2 ** 31) == native.ERR_UNSUPPORTED
    assert grouped(native, R=0) == native.OK
    assert grouped(native, N=0) == native.OK
    assert native.lib().tmg_grouped_gemm(None, None) == native.ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(M=-1), dict(activation=4), dict(activation=-1), dict(in_dtype=9), dict(ldd=8),
                                  dict(preact=16, ld_preact=3), dict(residual=16, ld_residual=-16), dict(D=None),
                                  dict(A=None), dict(b_row=-1)])
def test_linear_refuses(native, over):
    assert linear(native, **over) == native.ERR_INVALID_ARG


def test_linear_unsupported_and_empty(native):
    assert linear(native, in_dtype=native.F32) == native.ERR_UNSUPPORTED
    assert linear(native, M=0) == native.OK
    assert linear(native, N=0) == native.OK
    assert native.lib().tmg_linear(None, None) == native.ERR_INVALID_ARG


def test_wgrad_refuses(native):
    f = native.lib().tmg_grouped_gemm_wgrad
    good = [16, 16, 1, 16, 64, 1, 16, 16, None, 8, 16, 64, 2, 8]
    for at, v in ((9, -1), (10, -1), (11, -1), (12, 0), (12, 1025), (1, -16), (0, None), (3, None), (6, None), (7, None)):
        args = list(good)
        args[at] = v
        assert f(*args, None) == native.ERR_INVALID_ARG
    assert f(16, 16, 1, 16, 64, 1, 16, 16, None, 8, 0, 64, 2, 8, None) == native.OK


def test_linear_backward_refuses(native):
    f = native.lib().tmg_linear_backward
    good = [16, 16, 16, 16, 16, 64, 16, 64, 16, 16, 16, 8, 16, 64, 2]
    for at, v in ((0, None), (2, None), (4, None), (6, None), (11, -1), (14, 4), (14, -1), (1, -1), (7, -1)):
        args = list(good)
        args[at] = v
        assert f(*args, None) == native.ERR_INVALID_ARG


def test_routing_refuses(native):
    L = native.lib()
    route = [16, 4, 8, 2, 8, native.F32, 1, 16, 16, 16, 16, 16]
    for at, v in ((0, None), (1, -1), (2, 0), (2, 1025), (3, 0), (3, 9), (4, 7), (5, native.E4M3), (7, None), (9, None)):
        args = list(route)
        args[at] = v
        assert L.tmg_moe_route(*args, None) == native.ERR_INVALID_ARG
    back = [16, 4, 8, 2, 8, native.F32, 1, 16, 16, 16]
    for at, v in ((0, None), (1, -1), (3, 17), (5, 2), (7, None), (8, None), (9, None)):
        args = list(back)
        args[at] = v
        assert L.tmg_moe_route_backward(*args, None) == native.ERR_INVALID_ARG
    combine = [16, 8, 16, 16, 16, None, 0, 16, 16, 4, 16, 2]
    for at, v in ((0, None), (1, -1), (3, None), (7, None), (8, 15), (9, -1), (11, 0), (11, 17), (2, -1)):
        args = list(combine)
        args[at] = v
        assert L.tmg_moe_combine(*args, None) == native.ERR_INVALID_ARG
    grad = [16, 16, 16, 8, 16, 16, 16, 16, 16, 4, 16, 2]
    for at, v in ((0, None), (2, None), (5, None), (7, None), (9, -1), (11, 17)):
        args = list(grad)
        args[at] = v
        assert L.tmg_moe_combine_backward(*args, None) == native.ERR_INVALID_ARG
    assert L.tmg_moe_combine(16, 8, 16, 16, 16, None, 0, 16, 16, 0, 16, 2, None) == native.OK
