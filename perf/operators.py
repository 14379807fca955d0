"""The operators of a mixture-of-experts layer and of a dense projection, as measured cases.

Routing (``moe_route``, ``moe_combine`` and their gradients), matrix products grouped by
expert (``grouped_gemm``, ``grouped_gemm_wgrad``) and the dense product with bias,
activation and residual (``linear``, ``linear_backward``).  Each case is one call, or the
calls of one training step of one operator, at sizes that serving and training meet.
"""
import math

import torch

own = False

BF16, E4M3, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32


def listed():
    return [
        # the router of one decoding step of a small serving batch: latency only
        dict(name="route_step", op="route", T=5, E=64, k=8, normalize=True, dtype="f32", masked=False, grad=False),
        # the router of a training batch, with its gradient; experts masked off, padded tokens, bf16 ties
        dict(name="route_train", op="route", T=16381, E=128, k=8, normalize=True, dtype="bf16", masked=True, grad=True),
        # one token decoded: its eight experts' gate and up products, bound by reading their weights
        dict(name="grouped_step", op="up", T=1, E=64, k=8, H=2048, F=1024, dtype="bf16", train=False),
        # a serving batch of 61 sequences: a few rows for nearly every expert, the down product
        dict(name="grouped_batch", op="down", T=61, E=64, k=8, H=2048, F=1024, dtype="bf16", train=False),
        # prefill or training, ragged groups of about a thousand rows: gather, gate and up products, SwiGLU
        dict(name="grouped_train", op="up", T=8191, E=64, k=8, H=2048, F=1024, dtype="bf16", train=True),
        # prefill with 8-bit weights and activations, scales by token and by output column
        dict(name="grouped_e4m3", op="up", T=8192, E=32, k=4, H=4096, F=2048, dtype="e4m3", train=False),
        # the gradients of the down product: through SwiGLU to the gate and up products, and of the weights
        dict(name="grouped_backward", op="down_backward", T=8191, E=64, k=8, H=2048, F=1024, dtype="bf16", train=True),
        # the experts' answers weighted and added to the residual stream, prefill
        dict(name="combine_prefill", op="combine", T=8191, k=8, H=4096, residual=True),
        # its gradient in training
        dict(name="combine_backward", op="combine_backward", T=8191, k=8, H=4096),
        # a projection of a decoding step with bias, SiLU and residual, bound by reading its weight
        dict(name="linear_step", op="linear", M=16, N=8192, K=8192, act="silu", residual=True, train=False, dtype="bf16"),
        # a training forward with bias, GELU and residual that keeps what the gradient needs
        dict(name="linear_train", op="linear", M=8191, N=4096, K=4096, act="gelu", residual=True, train=True, dtype="bf16"),
        # its gradients: input, weight and bias
        dict(name="linear_backward", op="linear_backward", M=8191, N=4096, K=4096, act="gelu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "up", "up", "down", "down_backward", "up_backward", "combine", "combine_backward",
                     "linear", "linear", "linear_backward"])
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256])
        return dict(op=op, T=_log(rng, 1, 32768), E=E, k=rng.randint(1, 8), normalize=rng.random() < 0.6,
                    dtype=rng.choice(["f32", "bf16"]), masked=rng.random() < 0.5, grad=rng.random() < 0.5)
    if op in ("up", "down", "down_backward", "up_backward"):
        E = rng.choice([8, 16, 32, 64, 128])
        k = rng.randint(1, min(8, E // 2))
        dtype = "e4m3" if op in ("up", "down") and rng.random() < 0.3 else "bf16"
        step = 16 if dtype == "e4m3" else 8
        H = step * rng.randint(512 // step, 4096 // step)
        F = step * rng.randint(256 // step, 2048 // step)
        T = _log(rng, 64 if op.endswith("backward") else 1, 8192)
        T = max(1, min(T, int(2.0e11 / (2.0 * k * H * F))))
        return dict(op=op, T=T, E=E, k=k, H=H, F=F, dtype=dtype,
                    train=op.endswith("backward") or (dtype == "bf16" and op == "up" and rng.random() < 0.5))
    if op in ("combine", "combine_backward"):
        H, k = 8 * rng.randint(64, 512), rng.randint(1, 8)
        case = dict(op=op, T=_log(rng, 1, 8192), k=k, H=H)
        if op == "combine":
            case["residual"] = rng.random() < 0.5
        return case
    act = rng.choice(["none", "relu", "silu", "gelu"])
    N, K = 8 * rng.randint(64, 1024), 8 * rng.randint(64, 1024)
    if op == "linear_backward":
        M = max(1, min(_log(rng, 64, 8192), int(1.3e11 / (N * K))))
        return dict(op=op, M=M, N=N, K=K, act=act)
    dtype = rng.choice(["bf16", "bf16", "e4m3"])
    if dtype == "e4m3":
        K = K // 16 * 16
    M = max(1, min(_log(rng, 1, 8192), int(1.3e11 / (N * K))))
    return dict(op=op, M=M, N=N, K=K, act=act, residual=rng.random() < 0.5,
                train=dtype == "bf16" and rng.random() < 0.4, dtype=dtype)


# ------------------------------------------------------------------ inputs

def _router(T, E, g, skew=0.5):
    """Router logits with a preference for some experts, as trained routers have."""
    return torch.randn(T, E, generator=g, device="cuda") + skew * torch.randn(1, E, generator=g, device="cuda")


def _plan(T, E, k, g):
    """Routing of T tokens: offsets (E+1), rows (T*k) and the largest group."""
    top = _router(T, E, g).topk(k, dim=1).indices.reshape(-1)
    order = top.argsort(stable=True)
    counts = torch.bincount(top, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(T * k, device="cuda")
    return dict(offsets=offsets, rows=(order // k).to(torch.int32), slots=slots.view(T, k).to(torch.int32),
                most=int(counts.max()))


def _normal(shape, g, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _eight_bits(shape, g):
    """E4M3 values over most of the format's range and the fp32 scale of each row that brings them to order one."""
    x = torch.randn(shape, generator=g, device="cuda")
    top = x.abs().amax(-1, keepdim=True)
    return (x * (448.0 / top)).to(E4M3), (top[..., 0] / 448.0).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    op = case["op"]
    s = dict(case=dict(case), op=op)
    if op == "route":
        T, E = case["T"], case["E"]
        x = _router(T, E, g)
        if case["masked"]:
            # a tenth of the tokens are padding; every token may use about nine tenths of the experts
            x[torch.rand(T, E, generator=g, device="cuda") < 0.1] = -math.inf
            x[torch.rand(T, generator=g, device="cuda") < 0.1] = -math.inf
        s["logits"] = x.to(F32 if case["dtype"] == "f32" else BF16)
        s["dweights"] = torch.randn(T, case["k"], generator=g, device="cuda")
        return s
    if op in ("up", "down", "down_backward", "up_backward"):
        T, E, k, H, F = (case[n] for n in "TEkHF")
        s.update(_plan(T, E, k, g))
        R = T * k
        if op == "up" and case["dtype"] == "e4m3":
            s["A"], s["scale_a"] = _eight_bits((T, H), g)
            s["B"], s["scale_b"] = _eight_bits((E, 2 * F, H), g)
            s["scale_b"] /= math.sqrt(H)
        elif op == "down" and case["dtype"] == "e4m3":
            s["A"], s["scale_a"] = _eight_bits((R, F), g)
            s["B"], s["scale_b"] = _eight_bits((E, H, F), g)
            s["scale_b"] /= math.sqrt(F)
        elif op == "up":
            s["A"] = _normal((T, H), g)
            s["B"] = _normal((E, 2 * F, H), g, H ** -0.5)
        elif op == "down":
            s["A"] = _normal((R, F), g, 0.6)
            s["B"] = _normal((E, H, F), g, F ** -0.5)
        elif op == "down_backward":
            s["preact"] = _normal((R, 2 * F), g)
            s["hidden"] = _normal((R, F), g, 0.6)
            s["B"] = _normal((E, H, F), g, F ** -0.5)
            s["dD"] = _normal((R, H), g)
        else:
            s["A"] = _normal((T, H), g)
            s["B"] = _normal((E, 2 * F, H), g, H ** -0.5)
            s["dD"] = _normal((R, 2 * F), g)
        return s
    if op in ("combine", "combine_backward"):
        T, k, H = case["T"], case["k"], case["H"]
        s.update(_plan(T, 64, k, g))
        s["weights"] = torch.randn(T, k, generator=g, device="cuda").softmax(1)
        s["Y"] = _normal((T * k, H), g)
        s["residual"] = _normal((T, H), g) if case.get("residual") else None
        if op == "combine_backward":
            s["dOut"] = _normal((T, H), g)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    s["bias"] = torch.randn(N, generator=g, device="cuda") * 0.1
    if case.get("dtype") == "e4m3":
        s["A"], s["scale_a"] = _eight_bits((M, K), g)
        s["B"], s["scale_b"] = _eight_bits((N, K), g)
        s["scale_b"] /= math.sqrt(K)
    else:
        s["A"], s["B"], s["scale_a"], s["scale_b"] = _normal((M, K), g), _normal((N, K), g, K ** -0.5), None, None
    s["residual"] = _normal((M, N), g) if case.get("residual") else None
    if op == "linear_backward":
        s["preact"], s["dD"] = _normal((M, N), g), _normal((M, N), g)
    return s


# ---------------------------------------------------------- the calls and their plain forms

def run(state):
    return (_calls if own else _plain)(state)


def _calls(s):
    import tiled_mma_atom_gb300 as tmg
    c, op = s["case"], s["op"]
    if op == "route":
        r = tmg.moe_route(s["logits"], c["k"], normalize=c["normalize"])
        if not c["grad"]:
            return tuple(r)
        return tuple(r) + (tmg.moe_route_backward(s["logits"], r.experts, s["dweights"], normalize=c["normalize"]),)
    if op == "up":
        preact = torch.empty(c["T"] * c["k"], 2 * c["F"], dtype=BF16, device="cuda") if c["train"] else None
        D = tmg.grouped_gemm(s["A"], s["B"], s["offsets"], rows=s["rows"], activation="swiglu", preact=preact,
                             scale_a=s.get("scale_a"), scale_b=s.get("scale_b"))
        return (D, preact) if c["train"] else D
    if op == "down":
        return tmg.grouped_gemm(s["A"], s["B"], s["offsets"], scale_a=s.get("scale_a"), scale_b=s.get("scale_b"))
    if op == "down_backward":
        dH = tmg.grouped_gemm(s["dD"], s["B"].transpose(1, 2), s["offsets"], activation="swiglu_grad",
                              preact=s["preact"])
        return dH, tmg.grouped_gemm_wgrad(s["dD"], s["hidden"], s["offsets"])
    if op == "up_backward":
        dA = tmg.grouped_gemm(s["dD"], s["B"].transpose(1, 2), s["offsets"])
        return dA, tmg.grouped_gemm_wgrad(s["dD"], s["A"], s["offsets"], rows=s["rows"])
    if op == "combine":
        return tmg.moe_combine(s["Y"], s["slots"], s["weights"], residual=s["residual"])
    if op == "combine_backward":
        return tmg.moe_combine_backward(s["dOut"], s["Y"], s["slots"], s["weights"])
    if op == "linear":
        preact = torch.empty(c["M"], c["N"], dtype=BF16, device="cuda") if c["train"] else None
        D = tmg.linear(s["A"], s["B"], bias=s["bias"], activation=c["act"], residual=s["residual"], preact=preact,
                       scale_a=s["scale_a"], scale_b=s["scale_b"])
        return (D, preact) if c["train"] else D
    return tmg.linear_backward(s["dD"], s["A"], s["B"], preact=s["preact"], activation=c["act"])


def _silu(x):
    return x / (1 + torch.exp(-x))


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return _silu(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _groups(s):
    """(E, most) row numbers of every group, and which of them are rows."""
    o = s["offsets"].long()
    at = o[:-1, None] + torch.arange(s["most"], device="cuda")
    return at, at < o[1:, None]


def _spread(x, at, there):
    """The groups of x's rows, each padded with zeros to the largest."""
    return x.float()[at * there] * there[..., None]


def _collect(y, at, there, R):
    out = torch.empty((R + 1, y.shape[-1]), device="cuda")
    out[torch.where(there, at, R)] = y
    return out[:R]


def _plain_route(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["logits"].float()
    top, at = torch.sort(x, dim=1, descending=True, stable=True)
    top, at = top[:, :k], at[:, :k]
    there = top > -math.inf
    e = torch.where(there, torch.exp(top - top[:, :1]), 0.0)
    total = e.sum(1, keepdim=True) if c["normalize"] else torch.where(x > -math.inf, torch.exp(x - top[:, :1]), 0.0).sum(1, keepdim=True)
    weights = torch.where(there, e / total, 0.0)
    to = torch.where(there, at, E).reshape(-1)
    order = torch.argsort(to, stable=True)
    number = torch.arange(T * k, device="cuda")
    offsets = (to[:, None] < torch.arange(E + 1, device="cuda")).sum(0)
    rows = torch.where(number < offsets[-1], order // k, -1)
    slots = torch.empty_like(order)
    slots[order] = number
    slots = torch.where(there, slots.view(T, k), -1)
    found = (weights, torch.where(there, at, -1).int(), offsets.int(), rows.int(), slots.int())
    if not c["grad"]:
        return found
    dw = torch.where(there, s["dweights"], 0.0)
    mean = (weights * dw).sum(1, keepdim=True)
    if c["normalize"]:
        dx = torch.zeros_like(x)
    else:
        dx = torch.where(x > -math.inf, -mean * torch.exp(x - top[:, :1]) / total, 0.0)
        mean = torch.zeros_like(mean)
    dx = dx.scatter_add(1, at, weights * (dw - mean))
    return found + (dx.to(s["logits"].dtype),)


def _plain(s):
    c, op = s["case"], s["op"]
    if op == "route":
        return _plain_route(s)
    if op in ("up", "down", "down_backward", "up_backward"):
        R, F = c["T"] * c["k"], c["F"]
        at, there = _groups(s)
        B = s["B"].float()
        if op in ("up", "down"):
            x = s["A"].float()
            if s.get("scale_a") is not None:
                x, B = x * s["scale_a"][:, None], B * s["scale_b"][..., None]
            from_rows = s["rows"].long()[at * there] if op == "up" else at
            z = torch.bmm(_spread(x, from_rows, there), B.transpose(1, 2))
            if op == "down":
                return _collect(z, at, there, R).to(BF16)
            z = _collect(z, at, there, R)
            D = (_silu(z[:, :F]) * z[:, F:]).to(BF16)
            return (D, z.to(BF16)) if c["train"] else D
        dD = _spread(s["dD"], at, there)
        dA = _collect(torch.bmm(dD, B), at, there, R)
        if op == "up_backward":
            x = _spread(s["A"], s["rows"].long()[at * there], there)
        else:
            x = _spread(s["hidden"], at, there)
            gate, up = s["preact"][:, :F].float(), s["preact"][:, F:].float()
            dA = torch.cat([dA * up * _act_grad(gate, "silu"), dA * _silu(gate)], 1)
        return dA.to(BF16), torch.bmm(dD.transpose(1, 2), x).to(BF16)
    if op == "combine":
        out = (s["weights"][..., None] * s["Y"].float()[s["slots"].long()]).sum(1)
        return (out + s["residual"].float() if s["residual"] is not None else out).to(BF16)
    if op == "combine_backward":
        at, d = s["slots"].long(), s["dOut"].float()
        dY = torch.empty((c["T"] * c["k"], c["H"]), device="cuda")
        dY[at] = s["weights"][..., None] * d[:, None]
        return dY.to(BF16), (s["Y"].float()[at] * d[:, None]).sum(2)
    if op == "linear":
        x, B = s["A"].float(), s["B"].float()
        if s["scale_a"] is not None:
            x, B = x * s["scale_a"][:, None], B * s["scale_b"][:, None]
        z = x @ B.T + s["bias"]
        D = _act(z, c["act"])
        D = (D + s["residual"].float() if s["residual"] is not None else D).to(BF16)
        return (D, z.to(BF16)) if c["train"] else D
    dz = s["dD"].float() * _act_grad(s["preact"].float(), c["act"])
    return (dz @ s["B"].float()).to(BF16), (dz.T @ s["A"].float()).to(BF16), dz.sum(0)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    W = torch.float64
    if op == "route":
        x = s["logits"].cpu().to(W)
        T, E, k = c["T"], c["E"], c["k"]
        weights = torch.zeros(T, k, dtype=W)
        key = x.clone()
        picked, p_all = [], None
        for j in range(k):
            best = key.argmax(1)          # the lowest index of the largest, by the loop below
            best = (key == key.gather(1, best[:, None])).to(torch.int64).argmax(1)
            picked.append((best, key.gather(1, best[:, None])[:, 0] > -math.inf))
            key[torch.arange(T), best] = -math.inf
        at = torch.stack([b for b, _ in picked], 1)
        ok = torch.stack([v for _, v in picked], 1)
        lx = x.gather(1, at)
        top = torch.where(torch.isfinite(x), x, -1e300).amax(1, keepdim=True)
        num = torch.where(ok, torch.exp(lx - top), torch.zeros((), dtype=W))
        all_e = torch.where(torch.isfinite(x), torch.exp(x - top), torch.zeros((), dtype=W))
        den = (num if c["normalize"] else all_e).sum(1, keepdim=True).clamp(min=1e-300)
        weights = num / den
        if not c["grad"]:
            return (weights, None, None, None, None)
        dw = s["dweights"].cpu().to(W) * ok
        dx = torch.zeros(T, E, dtype=W)
        dot = (weights * dw).sum(1, keepdim=True)
        if c["normalize"]:
            dx.scatter_add_(1, at, weights * dw - weights * dot)
        else:
            dx -= all_e / den * dot
            dx.scatter_add_(1, at, weights * dw)
        return (weights, None, None, None, None, dx)
    if op in ("up", "down", "down_backward", "up_backward"):
        F, R, o = c["F"], c["T"] * c["k"], s["offsets"].tolist()
        rows = s["rows"].long()
        one, two = [], []
        for e in range(c["E"]):
            b, r = s["B"][e].to(W), slice(o[e], o[e + 1])
            if op in ("up", "down"):
                a = s["A"][rows[r]].to(W) if op == "up" else s["A"][r].to(W)
                z = a @ b.T
                if s.get("scale_a") is not None:
                    sa = s["scale_a"].to(W)
                    z = z * (sa[rows[r]] if op == "up" else sa[r])[:, None] * s["scale_b"][e].to(W)
                if op == "down":
                    one.append(z)
                    continue
                one.append(z[:, :F] * torch.sigmoid(z[:, :F]) * z[:, F:])
                if c["train"]:
                    two.append(z)
                continue
            d = s["dD"][r].to(W)
            da = d @ b
            if op == "down_backward":
                gate, up = s["preact"][r, :F].to(W), s["preact"][r, F:].to(W)
                p = torch.sigmoid(gate)
                da = torch.cat([da * up * (p + gate * p * (1 - p)), da * gate * p], 1)
                a = s["hidden"][r].to(W)
            else:
                a = s["A"][rows[r]].to(W)
            one.append(da)
            two.append(d.T @ a)
        if op == "up":
            return (torch.cat(one), torch.cat(two)) if c["train"] else torch.cat(one)
        return torch.cat(one) if op == "down" else (torch.cat(one), torch.stack(two))
    if op in ("combine", "combine_backward"):
        T, k, H = c["T"], c["k"], c["H"]
        at, w = s["slots"].long(), s["weights"].to(W)
        if op == "combine":
            out = s["residual"].to(W) if s["residual"] is not None else torch.zeros(T, H, dtype=W, device="cuda")
            for j in range(k):
                out = out + w[:, j, None] * s["Y"][at[:, j]].to(W)
            return out
        dY = torch.zeros(T * k, H, dtype=W, device="cuda")
        dw = torch.zeros(T, k, dtype=W, device="cuda")
        d = s["dOut"].to(W)
        for j in range(k):
            dY[at[:, j]] = w[:, j, None] * d
            dw[:, j] = (d * s["Y"][at[:, j]].to(W)).sum(1)
        return dY, dw
    if op == "linear":
        z = s["A"].to(W) @ s["B"].to(W).T
        if s["scale_a"] is not None:
            z = z * s["scale_a"].to(W)[:, None] * s["scale_b"].to(W)
        z = z + s["bias"].to(W)
        y = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "silu": lambda v: v * torch.sigmoid(v),
             "gelu": lambda v: v * 0.5 * torch.erfc(-v / math.sqrt(2.0))}[c["act"]](z)
        if s["residual"] is not None:
            y = y + s["residual"].to(W)
        return (y, z) if c["train"] else y
    v = s["preact"].to(W)
    p = torch.sigmoid(v)
    slope = {"none": torch.ones_like(v), "relu": (v > 0).to(W), "silu": p + v * p * (1 - p),
             "gelu": 0.5 * torch.erfc(-v / math.sqrt(2.0)) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)}[c["act"]]
    dz = s["dD"].to(W) * slope
    return dz @ s["B"].to(W), dz.T @ s["A"].to(W), dz.sum(0)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    if op == "route":
        each = 4 if c["dtype"] == "f32" else 2
        T, k = c["T"], c["k"]
        plan = T * k * 16 + 4 * (c["E"] + 1)
        again = T * c["E"] * 2 * each + T * k * 8 if c["grad"] else 0
        return {"bytes": T * c["E"] * each + plan + again, "flops": 0}
    if op in ("up", "down", "down_backward", "up_backward"):
        T, E, k, H, F = (c[n] for n in "TEkHF")
        R, each = T * k, 1 if c["dtype"] == "e4m3" else 2
        used = E * (1 - (1 - k / E) ** T)       # experts with rows, if all are as likely
        if op == "up":
            return {"bytes": T * H * each + used * 2 * F * H * each + R * F * 2 * (3 if c["train"] else 1) + 4 * R,
                    "flops": 4.0 * R * F * H}
        if op == "down":
            return {"bytes": R * F * each + used * F * H * each + R * H * 2, "flops": 2.0 * R * F * H}
        if op == "down_backward":
            return {"bytes": R * H * 2 + (used + E) * F * H * 2 + R * F * 10, "flops": 4.0 * R * F * H}
        return {"bytes": R * F * 4 + T * H * 2 + (used + E) * F * H * 4 + R * H * 2, "flops": 8.0 * R * F * H}
    if op == "combine":
        T, k, H = c["T"], c["k"], c["H"]
        return {"bytes": T * k * (2 * H + 8) + T * H * (4 if c["residual"] else 2), "flops": 2.0 * T * k * H}
    if op == "combine_backward":
        T, k, H = c["T"], c["k"], c["H"]
        return {"bytes": T * k * (4 * H + 12) + T * H * 2, "flops": 3.0 * T * k * H}
    M, N, K = c["M"], c["N"], c["K"]
    if op == "linear":
        each = 1 if c["dtype"] == "e4m3" else 2
        return {"bytes": (M + N) * K * each + M * N * 2 * (1 + bool(c["residual"]) + bool(c["train"])) + 4 * N,
                "flops": 2.0 * M * N * K}
    return {"bytes": M * N * (4 if c["act"] != "none" else 2) + 2 * (M + N) * K * 2 + 4 * N, "flops": 4.0 * M * N * K}
