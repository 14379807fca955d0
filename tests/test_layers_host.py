"""Host-side checks of the expert layer and of the products with adapters (no GPU):
what they refuse before any device work, what is empty, and that the gradients' formulas
are the forward's."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def native():
    from tiled_mma_atom_gb300 import build
    build.build()
    from tiled_mma_atom_gb300 import _native
    return _native


def moe(native, **over):
    v = dict(x=16, logits=16, W1=16, W2=16, residual=None, out=16, T=4, H=64, F=32, E=8, k=2, ldx=64, ld_logits=8,
             ld_residual=0, ld_out=64, logits_dtype=native.F32, normalize=1)
    v.update(over)
    return native.lib().tmg_moe_layer(ctypes.byref(native.MoeArgs(**v)), None)


def lora(native, **over):
    v = dict(x=16, W=16, A=16, B=16, D=16, adapters=16, scales=None, bias=None, residual=None, u=None, M=4, N=64, K=32, r=8,
             L=2, ldx=32, ldw=32, ldd=64, ld_residual=0)
    v.update(over)
    return native.lib().tmg_lora_linear(ctypes.byref(native.LoraArgs(**v)), None)


def grad(native, **over):
    v = dict(dD=16, x=16, W=16, A=16, B=16, adapters=16, scales=None, u=16, dx=16, dA=16, dB=16, M=4, N=64, K=32, r=8, L=2,
             ldd=64, ldx=32, ldw=32)
    v.update(over)
    return native.lib().tmg_lora_linear_backward(ctypes.byref(native.LoraGradArgs(**v)), None)


def test_struct_layouts(native):
    assert ctypes.sizeof(native.MoeArgs) == 6 * 8 + 9 * 8 + 8 == len(native.pack_moe(*[0] * 17))
    assert ctypes.sizeof(native.LoraArgs) == 10 * 8 + 9 * 8 == len(native.pack_lora(*[0] * 19))
    assert ctypes.sizeof(native.LoraGradArgs) == 11 * 8 + 8 * 8 == len(native.pack_lora_grad(*[0] * 19))


@pytest.mark.parametrize("over", [dict(T=-1), dict(H=-1), dict(F=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=64, ld_logits=64, k=17),
                                  dict(logits_dtype=2), dict(logits_dtype=9), dict(ld_logits=7), dict(ldx=-1), dict(ld_out=63),
                                  dict(residual=16, ld_residual=-1), dict(x=None), dict(logits=None), dict(W1=None),
                                  dict(W2=None), dict(out=None), dict(ldx=2 ** 60)])
def test_moe_layer_refuses(native, over):
    assert moe(native, **over) == native.ERR_INVALID_ARG
    assert native.lib().tmg_last_error()


def test_moe_layer_unsupported_and_empty(native):
    assert moe(native, T=2 ** 31) == native.ERR_UNSUPPORTED
    assert moe(native, H=2 ** 31, ldx=2 ** 31, ld_out=2 ** 31) == native.ERR_UNSUPPORTED
    assert moe(native, F=2 ** 30) == native.ERR_UNSUPPORTED
    assert moe(native, T=0) == native.OK
    assert moe(native, H=0) == native.OK
    assert native.lib().tmg_moe_layer(None, None) == native.ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(M=-1), dict(N=-1), dict(K=-1), dict(r=0), dict(r=257), dict(L=0), dict(L=1025), dict(ldx=-1),
                                  dict(ldw=-1), dict(ldd=63), dict(residual=16, ld_residual=-1), dict(x=None), dict(W=None),
                                  dict(A=None), dict(B=None), dict(D=None), dict(adapters=None), dict(ldx=2 ** 60)])
def test_lora_refuses(native, over):
    assert lora(native, **over) == native.ERR_INVALID_ARG
    assert native.lib().tmg_last_error()


@pytest.mark.parametrize("over", [dict(M=-1), dict(N=-1), dict(K=-1), dict(r=0), dict(r=257), dict(L=0), dict(L=1025), dict(ldx=-1),
                                  dict(ldw=-1), dict(ldd=-1), dict(x=None), dict(W=None), dict(A=None), dict(B=None), dict(dD=None),
                                  dict(u=None), dict(adapters=None)])
def test_lora_gradient_refuses(native, over):
    assert grad(native, **over) == native.ERR_INVALID_ARG
    assert native.lib().tmg_last_error()


def test_lora_unsupported_and_empty(native):
    assert lora(native, M=2 ** 31) == native.ERR_UNSUPPORTED
    assert grad(native, N=2 ** 31) == native.ERR_UNSUPPORTED
    assert lora(native, M=0) == native.OK
    assert native.lib().tmg_lora_linear(None, None) == native.ERR_INVALID_ARG
    assert native.lib().tmg_lora_linear_backward(None, None) == native.ERR_INVALID_ARG


def test_gradient_formulas():
    """The gradients that the GPU tests compare with, against autograd and against differences, in 64 bits."""
    g = torch.Generator().manual_seed(1)
    M, N, K, r, L = 7, 5, 6, 3, 2

    def rand(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64)

    ids = torch.tensor([0, 1, -1, 0, 1, 1, 0])
    W, scales, dD = rand(N, K), rand(L), rand(M, N)
    x, A, B = (rand(*s).requires_grad_() for s in ((M, K), (L, r, K), (L, N, r)))

    def forward(x, A, B):
        rows = []
        for m, a in enumerate(ids.tolist()):
            rows.append(W @ x[m] + (scales[a] * (B[a] @ (A[a] @ x[m])) if a >= 0 else 0))
        return torch.stack(rows)

    assert torch.autograd.gradcheck(forward, (x, A, B))
    want = torch.autograd.grad(forward(x, A, B), (x, A, B), dD)
    dx, dA, dB = dD @ W, torch.zeros(L, r, K, dtype=W.dtype), torch.zeros(L, N, r, dtype=W.dtype)
    for a in range(L):
        m = ids == a
        dU, u = scales[a] * (dD[m] @ B[a]), scales[a] * (x[m] @ A[a].T)
        dx[m] += dU @ A[a]
        dA[a], dB[a] = dU.T @ x[m], dD[m].T @ u
    for got, w in zip((dx, dA, dB), want):
        assert torch.allclose(got, w)


def _source(name):
    import os
    import re
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_mma_atom_gb300", "csrc", name)) as f:
        return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", f.read()))


@pytest.mark.parametrize("name,kernel", [("lora_few.cu", "lora_few_rank_kernel(RankArgs"), ("lora_rank.cu", "lora_rank_kernel(const"),
                                         ("lora_grad.cu", "lora_plan_kernel(const"), ("moe_few.cu", "moe_few_up_kernel(const")])
def test_successors_start_after_the_wait(name, kernel):
    """Kernels whose successor reads the call's inputs without a wait of its own let it start only after their own
    wait for the kernel before."""
    body = _source(name).split(kernel)[1]
    assert 0 < body.index("grid_wait();") < body.index("grid_release();")


@pytest.mark.parametrize("name,kernel", [("lora_few.cu", "lora_few_kernel(const"), ("lora_split.cu", "lora_split_kernel(const"),
                                         ("lora_pair.cu", "lora_pair_kernel(const"), ("moe_few.cu", "moe_few_down_kernel(const")])
def test_late_waits_are_every_warps(name, kernel):
    """Kernels that start beside the one before them end after it: every warp waits for it."""
    body = _source(name).split(kernel)[1].split("template <")[0]
    depth, found = 0, False
    for part in body.replace("{", " { ").replace("}", " } ").split(" "):
        depth += part == "{"
        depth -= part == "}"
        found |= depth == 1 and part == "grid_wait();"
    assert found


def test_kernels_settle_after_giving_up():
    """A kernel whose wait ran out leaves only when its loads have landed and its MMAs have run."""
    for name, loads, mmas in (("lora_pair.cu", "settle(full,", "settle(empty,"), ("lora_rank.cu", "settle(full,", "settle(done,"),
                              ("lora_split.cu", "settle(full,", "settle(done,"), ("lora_grad.cu", "settle(full,", "settle(empty,"),
                              ("few.cuh", "settle(sm.full,", "settle(&sm.done,"), ("moe_few.cu", "settle(sm.full,", "settle(sm.empty,"),
                              ("lora_few.cu", "settle(&bars[d],", "few_product(")):
        text = _source(name)
        assert loads in text and mmas in text, name
