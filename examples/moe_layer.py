"""A transformer block's feed-forward half with a mixture of experts, forward and
backward, on the library's operators:

    g = x · Wrᵀ                                   router logits (gemm)
    r = moe_route(g, k)                           experts, weights, row plan
    h = swiglu(x[rows] · W1[e]ᵀ)                  grouped_gemm, gather + SwiGLU
    y = h · W2[e]ᵀ                                grouped_gemm
    u = x + sum_j weights[t, j] y[slots[t, j]]    moe_combine with the residual
    v = u + gelu(u · Waᵀ + ba) · Wbᵀ + bb         linear, twice: a dense adapter

``python examples/moe_layer.py`` runs a training step and a single-token step
and prints their times.  Nothing waits for the GPU between the calls: the
plan of the grouped products stays there.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tiled_mma_atom_gb300 as tmg  # noqa: E402


class MoeBlock:
    """Parameters in bfloat16 on the GPU; H: model width, F: expert width, E
    experts of which each token takes k, A: adapter width."""

    def __init__(self, H: int, F: int, E: int, k: int, A: int, *, normalize: bool = True, seed: int = 0):
        g = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g) * shape[-1] ** -0.5).to(torch.bfloat16).cuda()

        self.k, self.normalize = k, normalize
        self.router, self.W1, self.W2 = weight(E, H), weight(E, 2 * F, H), weight(E, H, F)
        self.Wa, self.Wb = weight(A, H), weight(H, A)
        self.ba, self.bb = torch.zeros(A, device="cuda"), torch.zeros(H, device="cuda")

    def forward(self, x: torch.Tensor, train: bool = False):
        """x (T, H) bfloat16 -> (v, what backward needs)."""
        T, A = x.shape[0], self.Wa.shape[0]
        logits = tmg.gemm(x, self.router)
        r = tmg.moe_route(logits, self.k, normalize=self.normalize)

        def room(rows, cols):
            return torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda") if train else None

        pre1, pre2 = room(T * self.k, self.W1.shape[1]), room(T, A)
        h = tmg.grouped_gemm(x, self.W1, r.offsets, rows=r.rows, activation="swiglu", preact=pre1)
        y = tmg.grouped_gemm(h, self.W2, r.offsets)
        u = tmg.moe_combine(y, r.slots, r.weights, residual=x)
        a = tmg.linear(u, self.Wa, bias=self.ba, activation="gelu", preact=pre2)
        v = tmg.linear(a, self.Wb, bias=self.bb, residual=u)
        return v, (x, logits, r, pre1, h, y, u, pre2, a)

    def backward(self, dv: torch.Tensor, saved):
        """dv (T, H) bfloat16 -> dx and the parameters' gradients."""
        x, logits, r, pre1, h, y, u, pre2, a = saved
        da, dWb, dbb = tmg.linear_backward(dv, a, self.Wb)
        du, dWa, dba = tmg.linear_backward(da, u, self.Wa, preact=pre2, activation="gelu")
        du += dv                                                     # the adapter's residual
        dy, dweights = tmg.moe_combine_backward(du, y, r.slots, r.weights)
        dpre = tmg.grouped_gemm(dy, self.W2.transpose(1, 2), r.offsets, activation="swiglu_grad", preact=pre1)
        dW2 = tmg.grouped_gemm_wgrad(dy, h, r.offsets)
        dxr = tmg.grouped_gemm(dpre, self.W1.transpose(1, 2), r.offsets)
        dW1 = tmg.grouped_gemm_wgrad(dpre, x, r.offsets, rows=r.rows)
        dx = tmg.moe_combine(dxr, r.slots, residual=du)              # the gather's gradient, and the residual
        dlogits = tmg.moe_route_backward(logits, r.experts, dweights, normalize=self.normalize)
        dxg, drouter, _ = tmg.linear_backward(dlogits, x, self.router)
        dx += dxg
        return dx, dict(router=drouter, W1=dW1, W2=dW2, Wa=dWa, ba=dba, Wb=dWb, bb=dbb)


def _time(f, n=20):
    for _ in range(3):
        f()
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(n):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / n * 1e3


def main():
    H, F, E, k, A, T = 2048, 1024, 64, 8, 4096, 8192
    block = MoeBlock(H, F, E, k, A)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    dv = torch.randn(T, H, device="cuda").to(torch.bfloat16)

    def step():
        v, saved = block.forward(x, train=True)
        return block.backward(dv, saved)

    flops = 6.0 * T * (3 * k * H * F + 2 * H * A)
    us = _time(step)
    print(f"training step, {T} tokens: {us:.0f} us, {flops / us / 1e6:.0f} TFLOP/s")
    token = x[:1]
    print(f"one token, forward: {_time(lambda: block.forward(token)):.1f} us")
    tmg.check()


if __name__ == "__main__":
    main()
