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
from .grouped import _LOGITS, _bf16, _check, _current, _empty, _f32, _flat, _handle, _i32, _matrix, _side


def _run(call, args, stream, dev):
    """The library call, with the tensors' device current (a launch needs it)."""
    if torch.cuda.current_device() == dev.index:
        st = call(args, stream)
    else:
        with torch.cuda.device(dev):
            st = call(args, stream)
    if st:
        _native.raise_on(st)


def moe_layer(x: torch.Tensor, logits: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, k: int, *,
              normalize: bool = True, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """out[t] = residual[t] + sum over the k experts e of token t of
    w[t, e] * W2[e] · swiglu(W1[e] · x[t]), the whole expert layer in one call.

    x (T, H) bfloat16; logits (T, E) float32 or bfloat16, from which experts and
    weights are chosen as by moe_route (`normalize` as there); W1 (E, 2F, H) and
    W2 (E, H, F) bfloat16, contiguous; residual (T, H) bfloat16 (out itself is
    allowed).  The same as moe_route, grouped_gemm with SwiGLU, grouped_gemm and
    moe_combine, which it runs for many tokens; training takes those, since the
    gradients need what lies between them."""
    T, H = _matrix("x", x)
    E = _matrix("logits", logits)[1]
    F = _matrix("W2", W2, 3)[2]
    dt = _LOGITS.get(logits.dtype)
    if dt is None:
        raise TypeError(f"unsupported logits dtype {logits.dtype}: use float32 or bfloat16")
    dev = x.device
    side = None if stream is None else _side(stream, dev)
    _check("x", x, _bf16, (T, H))
    _check("logits", logits, logits.dtype, (T, E), dev)
    w1, w2 = _flat("W1", W1, _bf16, (E, 2 * F, H), dev), _flat("W2", W2, _bf16, (E, H, F), dev)
    if residual is not None:
        _check("residual", residual, _bf16, (T, H), dev)
    if out is None:
        out = _empty(side)((T, H), dtype=_bf16, device=dev)
    else:
        _check("out", out, _bf16, (T, H), dev)
    a = _native.pack_moe(x.data_ptr(), logits.data_ptr(), w1, w2, 0 if residual is None else residual.data_ptr(),
                         out.data_ptr(), T, H, F, E, k, x.stride(0), logits.stride(0),
                         0 if residual is None else residual.stride(0), out.stride(0), dt, 1 if normalize else 0)
    s = _current(dev.index) if side is None else _handle(side, (x, logits, W1, W2, residual, out))
    _run(_native.lib().tmg_moe_layer, a, s, dev)
    return out


def _adapter_shapes(A, B, N, K, dev):
    L, r, _ = _matrix("A", A, 3)
    return L, r, _flat("A", A, _bf16, (L, r, K), dev), _flat("B", B, _bf16, (L, N, r), dev)


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
    M, K = _matrix("x", x)
    N = _matrix("W", W)[0]
    dev = x.device
    side = None if stream is None else _side(stream, dev)
    _check("x", x, _bf16, (M, K))
    _check("W", W, _bf16, (N, K), dev)
    L, r, a_ptr, b_ptr = _adapter_shapes(A, B, N, K, dev)
    if residual is not None:
        _check("residual", residual, _bf16, (M, N), dev)
    if D is None:
        D = _empty(side)((M, N), dtype=_bf16, device=dev)
    else:
        _check("D", D, _bf16, (M, N), dev)
    a = _native.pack_lora(x.data_ptr(), W.data_ptr(), a_ptr, b_ptr, D.data_ptr(), _flat("adapters", adapters, _i32, (M,), dev),
                          0 if scales is None else _flat("scales", scales, _f32, (L,), dev),
                          0 if bias is None else _flat("bias", bias, _f32, (N,), dev),
                          0 if residual is None else residual.data_ptr(),
                          0 if u is None else _flat("u", u, _bf16, (M, r), dev), M, N, K, r, L, x.stride(0), W.stride(0),
                          D.stride(0), 0 if residual is None else residual.stride(0))
    s = _current(dev.index) if side is None else _handle(side, (x, W, A, B, D, adapters, scales, bias, residual, u))
    _run(_native.lib().tmg_lora_linear, a, s, dev)
    return D


def lora_linear_backward(dD: torch.Tensor, x: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                         adapters: torch.Tensor, u: torch.Tensor, *, scales: torch.Tensor | None = None, stream=None):
    """Gradients of lora_linear, its W frozen: (dx, dA, dB) bfloat16 with
    dU[m] = bf16(scales[a] * dD[m]·B[a]), dx = dD·W + dU·A[a] (M, K),
    dA[l] = sum of dU[m]ᵀ·x[m] and dB[l] = sum of dD[m]ᵀ·u[m] over the rows m of
    adapter l (zeros without any), shaped as A and B.  u: as lora_linear saved
    it.  The residual's gradient is dD; for those of W and the bias there is
    linear_backward."""
    M, N = _matrix("dD", dD)
    K = _matrix("x", x)[1]
    dev = dD.device
    side = None if stream is None else _side(stream, dev)
    new = _empty(side)
    _check("dD", dD, _bf16, (M, N))
    _check("x", x, _bf16, (M, K), dev)
    _check("W", W, _bf16, (N, K), dev)
    L, r, a_ptr, b_ptr = _adapter_shapes(A, B, N, K, dev)
    of, u_ptr = _flat("adapters", adapters, _i32, (M,), dev), _flat("u", u, _bf16, (M, r), dev)
    dx = new((M, K), dtype=_bf16, device=dev)
    dA, dB = new((L, r, K), dtype=_bf16, device=dev), new((L, N, r), dtype=_bf16, device=dev)
    a = _native.pack_lora_grad(dD.data_ptr(), x.data_ptr(), W.data_ptr(), a_ptr, b_ptr, of,
                               0 if scales is None else _flat("scales", scales, _f32, (L,), dev), u_ptr, dx.data_ptr(),
                               dA.data_ptr(), dB.data_ptr(), M, N, K, r, L, dD.stride(0), x.stride(0), W.stride(0))
    s = _current(dev.index) if side is None else _handle(side, (dD, x, W, A, B, adapters, scales, u, dx, dA, dB))
    _run(_native.lib().tmg_lora_linear_backward, a, s, dev)
    return dx, dA, dB
