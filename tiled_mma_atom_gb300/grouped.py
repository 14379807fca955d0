"""Mixture-of-experts routing, the products grouped by expert, and the dense
product with bias, activation and residual: argument marshalling for the
calls of include/tmg.h.

A layer with E experts of width F on tokens x (T, H), weights W1 (E, 2F, H)
and W2 (E, H, F)::

    r = moe_route(logits, k)
    h = grouped_gemm(x, W1, r.offsets, rows=r.rows, activation="swiglu")
    y = moe_combine(grouped_gemm(h, W2, r.offsets), r.slots, r.weights, residual=x)

Shapes never depend on values: the plan stays on the GPU, and no call waits
for it.  A `stream` other than the current one (a torch stream or a raw handle)
must be made to wait for the inputs, and the current one for the results, by the
caller; the tensors are recorded on both, so their memory is not reused before
the work on them is done.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _native
from ._native import BF16, E4M3, F32

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4, "swiglu_grad": 5}
_INPUTS = {torch.bfloat16: BF16, torch.float8_e4m3fn: E4M3}
_LOGITS = {torch.float32: F32, torch.bfloat16: BF16}
_bf16, _f32, _i32 = torch.bfloat16, torch.float32, torch.int32
_current = torch._C._cuda_getCurrentRawStream


class Routing(NamedTuple):
    """What moe_route returns; all tensors on the GPU."""
    weights: torch.Tensor     # (T, k) float32
    experts: torch.Tensor     # (T, k) int32, -1: no expert left
    offsets: torch.Tensor     # (E + 1,) int32: expert e's rows are offsets[e] .. offsets[e+1] - 1
    rows: torch.Tensor        # (T * k,) int32: the token of each row, -1 past offsets[E]
    slots: torch.Tensor       # (T, k) int32: the row of each (token, choice), -1 where there is none


def _side(stream, dev):
    """The stream of a call as a torch stream, or None where it is the current one."""
    if not hasattr(stream, "cuda_stream"):       # a raw handle; 0 and 1 name the default stream
        handle = int(stream)
        stream = torch.cuda.default_stream(dev) if handle in (0, 1) else torch.cuda.ExternalStream(handle, dev)
    return None if stream.cuda_stream == _current(dev.index) else stream


def _empty(side):
    """torch.empty for the outputs of a call.  On another stream (`side`) they are that
    stream's memory, since the current one's may still be read by what is queued there,
    and recorded on the current stream, where the caller will use them."""
    if side is None:
        return torch.empty

    def empty(*shape, **kind):
        with torch.cuda.stream(side):
            t = torch.empty(*shape, **kind)
        t.record_stream(torch.cuda.current_stream(t.device))
        return t
    return empty


def _handle(side, tensors):
    """The handle of another stream, with the call's tensors recorded on it."""
    for t in tensors:
        if t is not None:
            t.record_stream(side)
    return side.cuda_stream


def _check(name, t, dtype, shape, device=None, inner=True):
    """A CUDA tensor of this dtype and shape (unit column stride when `inner`)."""
    if t.shape != shape or t.dtype is not dtype or not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a {dtype} CUDA tensor of shape {shape}"
                         f"{'' if device is None else f' on {device}'}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    if inner and t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name} needs a unit column stride, got strides {t.stride()}")
    return t


def _flat(name, t, dtype, shape, device):
    """The pointer of an optional contiguous tensor."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}")
    return t.data_ptr()


def _matrix(name, t, dims=2):
    if t.dim() != dims or not t.is_cuda:
        raise ValueError(f"{name} must be a {dims}-D CUDA tensor, got shape {tuple(t.shape)} on {t.device}")
    return t.shape


def moe_route(logits: torch.Tensor, k: int, *, normalize: bool = True, stream=None) -> Routing:
    """Choose the k largest logits of each token and plan the grouped products.

    logits (T, E): float32 or bfloat16.  Equal logits go to the lower expert;
    -inf and NaN are never chosen.  normalize: weights are the softmax over the
    chosen logits, else the softmax over all of them."""
    T, E = _matrix("logits", logits)
    dt = _LOGITS.get(logits.dtype)
    if dt is None:
        raise TypeError(f"unsupported logits dtype {logits.dtype}: use float32 or bfloat16")
    if logits.stride(1) != 1:
        _check("logits", logits, logits.dtype, (T, E))
    dev = logits.device
    side = None if stream is None else _side(stream, dev)
    new = _empty(side)
    weights, experts = new((T, k), dtype=_f32, device=dev), new((T, k), dtype=_i32, device=dev)
    offsets, rows = new(E + 1, dtype=_i32, device=dev), new(T * k, dtype=_i32, device=dev)
    slots = new((T, k), dtype=_i32, device=dev)
    s = _current(dev.index) if side is None else _handle(side, (logits, weights, experts, offsets, rows, slots))
    st = _native.lib().tmg_moe_route(logits.data_ptr(), T, E, k, logits.stride(0), dt, 1 if normalize else 0,
                                     weights.data_ptr(), experts.data_ptr(), offsets.data_ptr(), rows.data_ptr(),
                                     slots.data_ptr(), s)
    if st:
        _native.raise_on(st)
    return Routing(weights, experts, offsets, rows, slots)


def moe_route_backward(logits: torch.Tensor, experts: torch.Tensor, dweights: torch.Tensor, *,
                       normalize: bool = True, stream=None) -> torch.Tensor:
    """Gradient of the logits given that of moe_route's weights; `experts` as
    moe_route returned them, `normalize` as it was called with."""
    T, E = _matrix("logits", logits)
    dt = _LOGITS.get(logits.dtype)
    if dt is None:
        raise TypeError(f"unsupported logits dtype {logits.dtype}: use float32 or bfloat16")
    if logits.stride(1) != 1:
        _check("logits", logits, logits.dtype, (T, E))
    k = experts.shape[-1]
    dev = logits.device
    side = None if stream is None else _side(stream, dev)
    new = _empty(side)
    d = new((T, E), dtype=logits.dtype, device=dev)
    s = _current(dev.index) if side is None else _handle(side, (logits, experts, dweights, d))
    st = _native.lib().tmg_moe_route_backward(logits.data_ptr(), T, E, k, logits.stride(0), dt, 1 if normalize else 0,
                                              _flat("experts", experts, _i32, (T, k), dev),
                                              _flat("dweights", dweights, _f32, (T, k), dev), d.data_ptr(), s)
    if st:
        _native.raise_on(st)
    return d


def moe_combine(Y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None, *,
                residual: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = residual[t] + sum over j of weights[t, j] * Y[slots[t, j]].

    Y (R, H) bfloat16; slots (T, k) int32, -1 adds nothing; weights (T, k)
    float32 or None (ones: the gradient of the gather by `rows`)."""
    R, H = _matrix("Y", Y)
    T, k = _matrix("slots", slots)
    dev = Y.device
    side = None if stream is None else _side(stream, dev)
    new = _empty(side)
    _check("Y", Y, _bf16, (R, H))
    if residual is not None:
        _check("residual", residual, _bf16, (T, H), dev)
    if out is None:
        out = new((T, H), dtype=_bf16, device=dev)
    else:
        _check("out", out, _bf16, (T, H), dev)
    s = _current(dev.index) if side is None else _handle(side, (Y, slots, weights, residual, out))
    st = _native.lib().tmg_moe_combine(Y.data_ptr(), R, Y.stride(0), _flat("slots", slots, _i32, (T, k), dev),
                                       _flat("weights", weights, _f32, (T, k), dev),
                                       None if residual is None else residual.data_ptr(),
                                       0 if residual is None else residual.stride(0), out.data_ptr(), out.stride(0),
                                       T, H, k, s)
    if st:
        _native.raise_on(st)
    return out


def moe_combine_backward(dOut: torch.Tensor, Y: torch.Tensor, slots: torch.Tensor,
                         weights: torch.Tensor | None = None, *, stream=None):
    """Gradients of moe_combine: (dY, dweights).  dY (R, H) bfloat16: rows that
    no slot names are left unwritten.  dweights (T, k) float32.  The residual's
    gradient is dOut."""
    T, H = _matrix("dOut", dOut)
    R, _ = _matrix("Y", Y)
    dev = dOut.device
    side = None if stream is None else _side(stream, dev)
    new = _empty(side)
    _check("dOut", dOut, _bf16, (T, H))
    _check("Y", Y, _bf16, (R, H), dev)
    k = slots.shape[-1]
    dY = new((R, H), dtype=_bf16, device=dev)
    dw = new((T, k), dtype=_f32, device=dev)
    s = _current(dev.index) if side is None else _handle(side, (dOut, Y, slots, weights, dY, dw))
    st = _native.lib().tmg_moe_combine_backward(dOut.data_ptr(), dOut.stride(0), Y.data_ptr(), R, Y.stride(0),
                                                _flat("slots", slots, _i32, (T, k), dev),
                                                _flat("weights", weights, _f32, (T, k), dev), dY.data_ptr(),
                                                dw.data_ptr(), T, H, k, s)
    if st:
        _native.raise_on(st)
    return dY, dw


def grouped_gemm(A: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor, D: torch.Tensor | None = None, *,
                 rows: torch.Tensor | None = None, activation: str = "none", preact: torch.Tensor | None = None,
                 scale_a: torch.Tensor | None = None, scale_b: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """D[r] = act(A[rows[r]] · B[e]ᵀ · scale_a[rows[r]] · scale_b[e]) for the rows
    offsets[e] <= r < offsets[e+1] of each expert e; rows in no group are left
    unwritten.

    A (T, K) and B (E, N, K): both bfloat16 or both float8_e4m3fn, any strides
    (``B.transpose(1, 2)`` of weights is read in place: the gradient of A).
    rows (R,) int32 or None (R = T).  scale_a (T,), scale_b (E, N) float32.
    activation: "none"; "swiglu": D (R, N/2) = silu(first half) * second half,
    the columns before it saved in preact (R, N) if given; "swiglu_grad": the
    product is the gradient of a SwiGLU result whose inputs are preact (R, 2N),
    D (R, 2N) their gradients."""
    T, K = _matrix("A", A)
    E, N, KB = _matrix("B", B, 3)
    dt = _INPUTS.get(A.dtype)
    if dt is None or B.dtype != A.dtype:
        raise TypeError(f"A and B must both be bfloat16 or both float8_e4m3fn, got {A.dtype} and {B.dtype}")
    dev = A.device
    side = None if stream is None else _side(stream, dev)
    new = _empty(side)
    if KB != K or B.device != dev:
        raise ValueError(f"B must be (E, N, {K}) on {dev}, got {tuple(B.shape)} on {B.device}")
    act = ACTIVATIONS.get(activation, -1)
    if act not in (0, 4, 5):
        raise ValueError(f"unknown activation {activation!r}; one of 'none', 'swiglu', 'swiglu_grad'")
    R = T if rows is None else rows.shape[0]
    cols, pcols = (N, 0) if act == 0 else (N // 2, N) if act == 4 else (2 * N, 2 * N)
    if act == 5 and preact is None:
        raise ValueError("swiglu_grad reads preact")
    if act and preact is not None:
        _check("preact", preact, _bf16, (R, pcols), dev)
    elif preact is not None:
        raise ValueError("preact goes with swiglu and swiglu_grad")
    if D is None:
        D = new((R, cols), dtype=_bf16, device=dev)
    else:
        _check("D", D, _bf16, (R, cols), dev)
    a = _native.pack_grouped(A.data_ptr(), B.data_ptr(), D.data_ptr(), _flat("offsets", offsets, _i32, (E + 1,), dev),
                             0 if rows is None else _flat("rows", rows, _i32, (R,), dev),
                             0 if scale_a is None else _flat("scale_a", scale_a, _f32, (T,), dev),
                             0 if scale_b is None else _flat("scale_b", scale_b, _f32, (E, N), dev),
                             0 if preact is None else preact.data_ptr(), R, N, K, E, T, *A.stride(), *B.stride(),
                             D.stride(0), 0 if preact is None else preact.stride(0), dt, act)
    s = _current(dev.index) if side is None else _handle(side, (A, B, offsets, rows, preact, scale_a, scale_b, D))
    st = _native.lib().tmg_grouped_gemm(a, s)
    if st:
        _native.raise_on(st)
    return D


def grouped_gemm_wgrad(dD: torch.Tensor, A: torch.Tensor, offsets: torch.Tensor, dB: torch.Tensor | None = None, *,
                       rows: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dB[e] = sum over the rows r of group e of dD[r]ᵀ · A[rows[r]]: the weight
    gradient of grouped_gemm, (E, N, K) bfloat16.  dD (R, N) and A (T, K)
    bfloat16; a group without rows gives zeros."""
    R, N = _matrix("dD", dD)
    T, K = _matrix("A", A)
    E = offsets.shape[0] - 1
    dev = dD.device
    side = None if stream is None else _side(stream, dev)
    new = _empty(side)
    _check("dD", dD, _bf16, (R, N), inner=False)
    _check("A", A, _bf16, (T, K), dev, inner=False)
    if rows is None and T != R:
        raise ValueError(f"without rows, A must have dD's {R} rows, got {T}")
    if dB is None:
        dB = new((E, N, K), dtype=_bf16, device=dev)
    s = _current(dev.index) if side is None else _handle(side, (dD, A, offsets, rows, dB))
    st = _native.lib().tmg_grouped_gemm_wgrad(dD.data_ptr(), *dD.stride(), A.data_ptr(), *A.stride(),
                                              _flat("dB", dB, _bf16, (E, N, K), dev),
                                              _flat("offsets", offsets, _i32, (E + 1,), dev),
                                              _flat("rows", rows, _i32, (R,), dev), R, N, K, E, T, s)
    if st:
        _native.raise_on(st)
    return dB


def linear(A: torch.Tensor, B: torch.Tensor, D: torch.Tensor | None = None, *, bias: torch.Tensor | None = None,
           activation: str = "none", residual: torch.Tensor | None = None, preact: torch.Tensor | None = None,
           scale_a: torch.Tensor | None = None, scale_b: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """D = bf16(act(z) + residual), z = A·Bᵀ · scale_a[m] · scale_b[n] + bias[n].

    A (M, K) and B (N, K): both bfloat16 or both float8_e4m3fn, any strides.
    bias (N,), scale_a (M,), scale_b (N,) float32; residual (M, N) bfloat16
    (D itself is allowed); preact (M, N) bfloat16: z is saved there for
    linear_backward.  activation: "none", "relu", "silu", "gelu" (erf form)."""
    M, K = _matrix("A", A)
    N, KB = _matrix("B", B)
    dt = _INPUTS.get(A.dtype)
    if dt is None or B.dtype != A.dtype:
        raise TypeError(f"A and B must both be bfloat16 or both float8_e4m3fn, got {A.dtype} and {B.dtype}")
    dev = A.device
    side = None if stream is None else _side(stream, dev)
    new = _empty(side)
    if KB != K or B.device != dev:
        raise ValueError(f"B must be (N, {K}) on {dev}, got {tuple(B.shape)} on {B.device}")
    act = ACTIVATIONS.get(activation, -1)
    if not 0 <= act <= 3:
        raise ValueError(f"unknown activation {activation!r}; one of 'none', 'relu', 'silu', 'gelu'")
    if D is None:
        D = new((M, N), dtype=_bf16, device=dev)
    else:
        _check("D", D, _bf16, (M, N), dev)
    if residual is not None:
        _check("residual", residual, _bf16, (M, N), dev)
    if preact is not None:
        _check("preact", preact, _bf16, (M, N), dev)
    a = _native.pack_linear(A.data_ptr(), B.data_ptr(), D.data_ptr(),
                            0 if scale_a is None else _flat("scale_a", scale_a, _f32, (M,), dev),
                            0 if scale_b is None else _flat("scale_b", scale_b, _f32, (N,), dev),
                            0 if bias is None else _flat("bias", bias, _f32, (N,), dev),
                            0 if residual is None else residual.data_ptr(), 0 if preact is None else preact.data_ptr(),
                            M, N, K, *A.stride(), *B.stride(), D.stride(0), 0 if residual is None else residual.stride(0),
                            0 if preact is None else preact.stride(0), dt, act)
    s = _current(dev.index) if side is None else _handle(side, (A, B, D, bias, residual, preact, scale_a, scale_b))
    st = _native.lib().tmg_linear(a, s)
    if st:
        _native.raise_on(st)
    return D


def linear_backward(dD: torch.Tensor, A: torch.Tensor, B: torch.Tensor, *, preact: torch.Tensor | None = None,
                    activation: str = "none", stream=None):
    """Gradients of linear (bfloat16, no scales): (dA, dB, dbias) with
    dz = dD * act'(preact), dA = dz·B (M, K), dB = dzᵀ·A (N, K) bfloat16 and
    dbias (N,) float32, the column sums of dz before its rounding to bfloat16.
    preact is needed unless activation is "none".  The residual's gradient is
    dD."""
    M, N = _matrix("dD", dD)
    K = _matrix("A", A)[1]
    dev = dD.device
    side = None if stream is None else _side(stream, dev)
    new = _empty(side)
    act = ACTIVATIONS.get(activation, -1)
    if not 0 <= act <= 3:
        raise ValueError(f"unknown activation {activation!r}; one of 'none', 'relu', 'silu', 'gelu'")
    _check("dD", dD, _bf16, (M, N))
    _check("A", A, _bf16, (M, K), dev)
    _check("B", B, _bf16, (N, K), dev)
    if act:
        if preact is None:
            raise ValueError(f"the gradient of {activation} reads preact")
        _check("preact", preact, _bf16, (M, N), dev)
    else:
        preact = None
    dA = new((M, K), dtype=_bf16, device=dev)
    dB = new((N, K), dtype=_bf16, device=dev)
    dbias = new((N,), dtype=_f32, device=dev)
    s = _current(dev.index) if side is None else _handle(side, (dD, A, B, preact, dA, dB, dbias))
    st = _native.lib().tmg_linear_backward(dD.data_ptr(), dD.stride(0), None if preact is None else preact.data_ptr(),
                                           0 if preact is None else preact.stride(0), A.data_ptr(), A.stride(0),
                                           B.data_ptr(), B.stride(0), dA.data_ptr(), dB.data_ptr(), dbias.data_ptr(),
                                           M, N, K, act, s)
    if st:
        _native.raise_on(st)
    return dA, dB, dbias
