"""The whole mixture-of-experts layer of a few tokens, and dense projections with low-rank
adapters, as measured cases.

``moe_layer`` routes tokens, runs their experts and adds up the answers in one call;
``lora_linear`` adds each row's own low-rank adapter to a shared projection, and
``lora_linear_backward`` gives the gradients of its input and of the adapters, the shared
weight being frozen.  Each case is one call, at sizes that serving and training meet.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


def listed():
    return [
        # one token decoded through an expert layer: eight of 64 experts, bound by reading their weights
        dict(name="moe_token", op="moe", T=1, E=64, k=8, H=2048, F=1024, normalize=True, dtype="f32", masked=False, residual=True),
        # a small serving batch of wider experts, logits in bf16 with ties, some sequences at their end (padding)
        dict(name="moe_few", op="moe", T=13, E=32, k=4, H=4096, F=2048, normalize=False, dtype="bf16", masked=True, residual=True),
        # 61 sequences decoded together: nearly every expert is in use
        dict(name="moe_batch", op="moe", T=61, E=64, k=8, H=2048, F=1024, normalize=True, dtype="f32", masked=False, residual=False),
        # one request's token through a projection with its adapter: latency
        dict(name="lora_token", op="lora", M=1, N=4096, K=4096, r=16, L=8, run=1, bias=False, residual=False),
        # sixteen requests decoded together, most with adapters of their own
        dict(name="lora_step", op="lora", M=16, N=8192, K=8192, r=16, L=64, run=1, bias=False, residual=True),
        # a full decoding batch with adapters of a higher rank
        dict(name="lora_batch", op="lora", M=61, N=4096, K=4096, r=64, L=32, run=1, bias=True, residual=False),
        # short prompts and single tokens in one batch, a narrow projection
        dict(name="lora_mixed", op="lora", M=700, N=1024, K=4096, r=32, L=16, run=50, bias=True, residual=False),
        # packed prompts of several requests, some of them without an adapter
        dict(name="lora_prompt", op="lora", M=8191, N=4096, K=4096, r=16, L=8, run=900, bias=False, residual=True),
        # the gradients of a small batch that trains two adapters of rank 64
        dict(name="lora_grad_small", op="lora_grad", M=700, N=4096, K=2048, r=64, L=2, run=300),
        # the gradients of a training batch, packed sequences of four tenants
        dict(name="lora_grad", op="lora_grad", M=8191, N=4096, K=4096, r=16, L=4, run=900),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["moe", "moe", "lora", "lora", "lora", "lora_grad"])
    if op == "moe":
        E = rng.choice([8, 16, 32, 60, 64, 128])
        return dict(op=op, T=_log(rng, 1, 64), E=E, k=rng.randint(1, min(8, E // 2)), H=8 * rng.randint(64, 512),
                    F=8 * rng.randint(32, 256), normalize=rng.random() < 0.6, dtype=rng.choice(["f32", "bf16"]),
                    masked=rng.random() < 0.4, residual=rng.random() < 0.6)
    N, K = 8 * rng.randint(64, 1024), 8 * rng.randint(64, 1024)
    r = rng.choice([4, 8, 16, 16, 32, 64, 128])
    L = _log(rng, 1, min(64, 2048 // r))
    M = max(1, min(_log(rng, 1 if op == "lora" else 64, 8192), int(1.3e11 / (N * K))))
    case = dict(op=op, M=M, N=N, K=K, r=r, L=L, run=1 if M <= 64 else _log(rng, 20, 2000))
    if op == "lora":
        case.update(bias=rng.random() < 0.4, residual=rng.random() < 0.4)
    return case


# ------------------------------------------------------------------ inputs

def _normal(shape, g, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _requests(M, L, run, g):
    """The adapter of each row: requests one after another, of `run` rows on average and
    between a fifth and nine fifths of that, one in seven without an adapter (-1)."""
    n = M if run == 1 else 8 + 2 * M // run
    length = torch.ones(n, device="cuda") if run == 1 else run * (0.2 + 1.6 * torch.rand(n, generator=g, device="cuda"))
    end = length.round().clamp(min=1).cumsum(0)
    end[-1] = max(M, n)
    of = torch.randint(0, L, (n,), generator=g, device="cuda")
    of = torch.where(torch.rand(n, generator=g, device="cuda") < 1 / 7, -1, of)
    return of[torch.searchsorted(end, torch.arange(M, device="cuda") + 0.5)].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 29)
    c, op = case, case["op"]
    s = dict(case=dict(case), op=op)
    if op == "moe":
        T, E, H, F = c["T"], c["E"], c["H"], c["F"]
        logits = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(1, E, generator=g, device="cuda")
        if c["masked"]:
            # a tenth of the tokens are padding; every token may use about nine tenths of the experts
            logits[torch.rand(T, E, generator=g, device="cuda") < 0.1] = -math.inf
            logits[torch.rand(T, generator=g, device="cuda") < 0.1] = -math.inf
        s["logits"] = logits.to(F32 if c["dtype"] == "f32" else BF16)
        s["x"] = _normal((T, H), g)
        s["W1"], s["W2"] = _normal((E, 2 * F, H), g, H ** -0.5), _normal((E, H, F), g, F ** -0.5)
        s["residual"] = _normal((T, H), g) if c["residual"] else None
        return s
    M, N, K, r, L = (c[n] for n in "MNKrL")
    s["adapters"] = _requests(M, L, c["run"], g)
    s["scales"] = 0.5 + 1.5 * torch.rand(L, generator=g, device="cuda")
    s["x"], s["W"] = _normal((M, K), g), _normal((N, K), g, K ** -0.5)
    s["A"], s["B"] = _normal((L, r, K), g, K ** -0.5), _normal((L, N, r), g, 0.5 * r ** -0.5)
    if op == "lora_grad":
        s["dD"], s["u"] = _normal((M, N), g), _normal((M, r), g)
        return s
    s["bias"] = torch.randn(N, generator=g, device="cuda") * 0.1 if c["bias"] else None
    s["residual"] = _normal((M, N), g) if c["residual"] else None
    return s


# ---------------------------------------------------------- the calls and their plain forms

def run(state):
    return (_calls if own else _plain)(state)


def _calls(s):
    import tiled_mma_atom_gb300 as tmg
    c = s["case"]
    if s["op"] == "moe":
        return tmg.moe_layer(s["x"], s["logits"], s["W1"], s["W2"], c["k"], normalize=c["normalize"], residual=s["residual"])
    if s["op"] == "lora":
        return tmg.lora_linear(s["x"], s["W"], s["A"], s["B"], s["adapters"], scales=s["scales"], bias=s["bias"],
                               residual=s["residual"])
    return tmg.lora_linear_backward(s["dD"], s["x"], s["W"], s["A"], s["B"], s["adapters"], s["u"], scales=s["scales"])


def _plain_moe(s):
    c = s["case"]
    T, E, k, F = c["T"], c["E"], c["k"], c["F"]
    g = s["logits"].float()
    top, at = torch.sort(g, dim=1, descending=True, stable=True)
    top, at = top[:, :k], at[:, :k]
    e = torch.where(top > -math.inf, torch.exp(top - top[:, :1]), 0.0)
    total = e.sum(1, keepdim=True) if c["normalize"] else torch.where(g > -math.inf, torch.exp(g - top[:, :1]), 0.0).sum(1, keepdim=True)
    w = torch.zeros(T, E, device="cuda").scatter(1, at, torch.where(top > -math.inf, e / total, 0.0))
    # every expert's product with every token; the weights are zero where it was not chosen
    z = (s["x"].float() @ s["W1"].float().view(E * 2 * F, -1).T).view(T, E, 2, F)
    h = z[:, :, 0] / (1 + torch.exp(-z[:, :, 0])) * z[:, :, 1] * w[..., None]
    out = torch.bmm(h.transpose(0, 1), s["W2"].float().transpose(1, 2)).sum(0)
    return (out + s["residual"].float() if s["residual"] is not None else out).to(BF16)


def _own_rank(wide, s):
    """Of (M, L r) products with all adapters, each row's own, as (M, L r) with zeros elsewhere, and scaled."""
    M, L = wide.shape[0], s["case"]["L"]
    mine = s["adapters"][:, None] == torch.arange(L, device="cuda")
    return (wide.view(M, L, -1) * (mine * s["scales"])[..., None]).view(M, -1)


def _plain(s):
    if s["op"] == "moe":
        return _plain_moe(s)
    c = s["case"]
    M, N, K, r, L = (c[n] for n in "MNKrL")
    x, A, B = s["x"].float(), s["A"].float().view(L * r, K), s["B"].float().transpose(1, 2).reshape(L * r, N)
    if s["op"] == "lora":
        D = x @ s["W"].float().T + _own_rank(x @ A.T, s) @ B
        if s["bias"] is not None:
            D = D + s["bias"]
        return (D + s["residual"].float() if s["residual"] is not None else D).to(BF16)
    dD = s["dD"].float()
    dU = _own_rank(dD @ B.T, s)
    mine = s["adapters"][:, None] == torch.arange(L, device="cuda")
    U = (s["u"].float()[:, None] * mine[..., None]).view(M, L * r)
    return ((dD @ s["W"].float() + dU @ A).to(BF16), (dU.T @ x).view(L, r, K).to(BF16),
            (dD.T @ U).view(N, L, r).transpose(0, 1).to(BF16).contiguous())


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    W = torch.float64
    if case["op"] == "moe":
        T, H, F = case["T"], case["H"], case["F"]
        x = s["x"].to(W)
        out = s["residual"].to(W) if s["residual"] is not None else torch.zeros(T, H, dtype=W, device="cuda")
        for t, row in enumerate(s["logits"].double().cpu().tolist()):
            chosen = sorted((e for e in range(case["E"]) if row[e] > -math.inf), key=lambda e: (-row[e], e))[:case["k"]]
            if not chosen:
                continue
            of = chosen if case["normalize"] else [e for e in range(case["E"]) if row[e] > -math.inf]
            total = sum(math.exp(row[e] - row[chosen[0]]) for e in of)
            for e in chosen:
                z = s["W1"][e].to(W) @ x[t]
                h = z[:F] * torch.sigmoid(z[:F]) * z[F:]
                out[t] += math.exp(row[e] - row[chosen[0]]) / total * (s["W2"][e].to(W) @ h)
        return out
    of, x = s["adapters"].long(), s["x"].to(W)
    rows = [(l, (of == l).nonzero()[:, 0], s["A"][l].to(W), s["B"][l].to(W), float(s["scales"][l])) for l in range(case["L"])]
    if case["op"] == "lora":
        D = x @ s["W"].to(W).T
        for _, m, A, B, scale in rows:
            D[m] += scale * ((x[m] @ A.T) @ B.T)
        if s["bias"] is not None:
            D += s["bias"].to(W)
        return D + s["residual"].to(W) if s["residual"] is not None else D
    dD, u = s["dD"].to(W), s["u"].to(W)
    dx = dD @ s["W"].to(W)
    dA, dB = torch.zeros_like(s["A"], dtype=W), torch.zeros_like(s["B"], dtype=W)
    for l, m, A, B, scale in rows:
        dU = scale * (dD[m] @ B)
        dx[m] += dU @ A
        dA[l] = dU.T @ x[m]
        dB[l] = dD[m].T @ u[m]
    return dx, dA, dB


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "moe":
        T, E, k, H, F = (c[n] for n in "TEkHF")
        used = E * (1 - (1 - k / E) ** T)       # experts in use, if all are as likely
        logits = T * E * (4 if c["dtype"] == "f32" else 2)
        return {"bytes": used * 3 * F * H * 2 + T * H * 2 * (3 if c["residual"] else 2) + logits, "flops": 6.0 * T * k * F * H}
    M, N, K, r, L = (c[n] for n in "MNKrL")
    requests = max(1, M / c["run"])
    used = L * (1 - (1 - 6 / 7 / L) ** requests)   # adapters in use, if all are as likely
    ranks = 2 * r * (N + K)
    if c["op"] == "lora":
        return {"bytes": 2 * (M + N) * K + 2 * M * N * (2 if c["residual"] else 1) + used * ranks + 4 * (M + (N if c["bias"] else 0)),
                "flops": 2.0 * M * N * K + 2.0 * M * r * (N + K)}
    return {"bytes": 2 * M * N + 4 * M * K + 2 * N * K + 2 * M * r + (used + L) * ranks + 4 * M,
            "flops": 2.0 * M * N * K + 4.0 * M * r * (N + K)}
