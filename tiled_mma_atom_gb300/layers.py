"""Calls that run several products: the whole mixture-of-experts layer, and the dense
product with low-rank adapters.  Argument marshalling for the calls of include/tmg.h.

One decoding step of a served model, every request with its own adapter::

    y = lora_linear(x, W, A, B, adapters, scales=scales)
    out = moe_layer(y, logits, W1, W2, k, residual=y)

Streams, workspaces and other devices: as in the calls of grouped.py.
"""
from __future__ import annotations

import torch

from . import _native
from .grouped import _LOGITS, _bf16, _current, _empty, _f32, _handle, _i32, _side

_device = torch._C._cuda_getDevice


def _run(call, args, stream, index):
    """The library call, with the tensors' device current (a launch needs it)."""
    if _device() == index:
        st = call(args, stream)
    else:
        with torch.cuda.device(index):
            st = call(args, stream)
    if st:
        _native.raise_on(st)


def _wrong(name, t, dtype, shape, index, what):
    raise ValueError(f"{name} must be a {what} {dtype} tensor of shape {tuple(shape)} on cuda:{index}, got {t.dtype} "
                     f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _rows(name, t, dtype, shape, index):
    """The pointer of a matrix on GPU `index` with unit column stride."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not (t.is_contiguous() or t.stride(1) == 1 or shape[1] <= 1):
        _wrong(name, t, dtype, shape, index, "row-wise contiguous")
    return t.data_ptr()


def _flat(name, t, dtype, shape, index):
    """The pointer of a contiguous tensor on GPU `index`."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        _wrong(name, t, dtype, shape, index, "contiguous")
    return t.data_ptr()


def _gpu(name, t, dims):
    """The number of the GPU of a tensor with `dims` dimensions."""
    index = t.get_device()
    if index < 0 or t.dim() != dims:
        raise ValueError(f"{name} must be a {dims}-D CUDA tensor, got shape {tuple(t.shape)} on {t.device}")
    return index


def _dims(name, t, dims):
    if t.dim() != dims:
        raise ValueError(f"{name} must be {dims}-D, got shape {tuple(t.shape)}")
    return t.shape


def moe_layer(x: torch.Tensor, logits: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, k: int, *,
              normalize: bool = True, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """out[t] = residual[t] + sum over the k experts e of token t of
    w[t, e] * W2[e] · swiglu(W1[e] · x[t]), the whole expert layer in one call.

    x (T, H) bfloat16; logits (T, E) float32 or bfloat16, from which experts and
    weights are chosen as by moe_route (`normalize` as there); W1 (E, 2F, H) and
    W2 (E, H, F) bfloat16, contiguous; residual (T, H) bfloat16 (out itself is
    allowed).  Up to 64 tokens the layer has kernels of its own; more run
    moe_route, grouped_gemm with SwiGLU, grouped_gemm and moe_combine.  Training
    takes those, since the gradients need what lies between them."""
    i = _gpu("x", x, 2)
    T, H = x.shape
    E = _dims("logits", logits, 2)[1]
    F = _dims("W2", W2, 3)[2]
    dt = _LOGITS.get(logits.dtype)
    if dt is None:
        raise TypeError(f"unsupported logits dtype {logits.dtype}: use float32 or bfloat16")
    side = None if stream is None else _side(stream, x.device)
    if out is None:
        out = _empty(side)((T, H), dtype=_bf16, device=x.device)
        to = out.data_ptr()
    else:
        to = _rows("out", out, _bf16, (T, H), i)
    a = _native.pack_moe(_rows("x", x, _bf16, (T, H), i), _rows("logits", logits, logits.dtype, (T, E), i),
                         _flat("W1", W1, _bf16, (E, 2 * F, H), i), _flat("W2", W2, _bf16, (E, H, F), i),
                         0 if residual is None else _rows("residual", residual, _bf16, (T, H), i),
                         to, T, H, F, E, k, x.stride(0), logits.stride(0),
                         0 if residual is None else residual.stride(0), out.stride(0), dt, 1 if normalize else 0)
    s = _current(i) if side is None else _handle(side, (x, logits, W1, W2, residual, out))
    _run(_native.lib().tmg_moe_layer, a, s, i)
    return out


def lora_linear(x: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, adapters: torch.Tensor,
                D: torch.Tensor | None = None, *, scales: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                residual: torch.Tensor | None = None, u: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """D[m] = x[m]·Wᵀ + u[m]·B[a]ᵀ + bias + residual[m] with a = adapters[m] and
    u[m] = bf16(scales[a] * x[m]·A[a]ᵀ): a projection shared by many requests, each
    row with the low-rank adapter of its request.

    x (M, K), W (N, K) bfloat16, unit column strides; A (L, r, K) and B (L, N, r)
    bfloat16, contiguous, r <= 256, L <= 1024 (pad adapters of lower rank with
    zeros); adapters (M,) int32, where -1 (or any number outside) is no adapter;
    scales (L,) and bias (N,) float32; residual (M, N) bfloat16 (D itself is
    allowed); u (M, r) bfloat16: u is saved there for lora_linear_backward."""
    i = _gpu("x", x, 2)
    M, K = x.shape
    N = _dims("W", W, 2)[0]
    L, r, _ = _dims("A", A, 3)
    side = None if stream is None else _side(stream, x.device)
    if D is None:
        D = _empty(side)((M, N), dtype=_bf16, device=x.device)
        to = D.data_ptr()
    else:
        to = _rows("D", D, _bf16, (M, N), i)
    a = _native.pack_lora(_rows("x", x, _bf16, (M, K), i), _rows("W", W, _bf16, (N, K), i), _flat("A", A, _bf16, (L, r, K), i),
                          _flat("B", B, _bf16, (L, N, r), i), to, _flat("adapters", adapters, _i32, (M,), i),
                          0 if scales is None else _flat("scales", scales, _f32, (L,), i),
                          0 if bias is None else _flat("bias", bias, _f32, (N,), i),
                          0 if residual is None else _rows("residual", residual, _bf16, (M, N), i),
                          0 if u is None else _flat("u", u, _bf16, (M, r), i), M, N, K, r, L, x.stride(0), W.stride(0),
                          D.stride(0), 0 if residual is None else residual.stride(0))
    s = _current(i) if side is None else _handle(side, (x, W, A, B, D, adapters, scales, bias, residual, u))
    _run(_native.lib().tmg_lora_linear, a, s, i)
    return D


def lora_linear_backward(dD: torch.Tensor, x: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                         adapters: torch.Tensor, u: torch.Tensor, *, scales: torch.Tensor | None = None, stream=None):
    """Gradients of lora_linear, its W frozen: (dx, dA, dB) bfloat16 with
    dU[m] = bf16(scales[a] * dD[m]·B[a]), dx = dD·W + dU·A[a] (M, K),
    dA[l] = sum of dU[m]ᵀ·x[m] and dB[l] = sum of dD[m]ᵀ·u[m] over the rows m of
    adapter l (zeros without any), shaped as A and B.  u: as lora_linear saved
    it.  The residual's gradient is dD; for those of W and the bias there is
    linear_backward."""
    i = _gpu("dD", dD, 2)
    M, N = dD.shape
    K = _dims("x", x, 2)[1]
    L, r, _ = _dims("A", A, 3)
    dev = dD.device
    side = None if stream is None else _side(stream, dev)
    new = _empty(side)
    dx = new((M, K), dtype=_bf16, device=dev)
    dA, dB = new((L, r, K), dtype=_bf16, device=dev), new((L, N, r), dtype=_bf16, device=dev)
    a = _native.pack_lora_grad(_rows("dD", dD, _bf16, (M, N), i), _rows("x", x, _bf16, (M, K), i), _rows("W", W, _bf16, (N, K), i),
                               _flat("A", A, _bf16, (L, r, K), i), _flat("B", B, _bf16, (L, N, r), i),
                               _flat("adapters", adapters, _i32, (M,), i),
                               0 if scales is None else _flat("scales", scales, _f32, (L,), i), _flat("u", u, _bf16, (M, r), i),
                               dx.data_ptr(), dA.data_ptr(), dB.data_ptr(), M, N, K, r, L, dD.stride(0), x.stride(0), W.stride(0))
    s = _current(i) if side is None else _handle(side, (dD, x, W, A, B, adapters, scales, u, dx, dA, dB))
    _run(_native.lib().tmg_lora_linear_backward, a, s, i)
    return dx, dA, dB
