"""Captured graphs whose kernels name workspaces (operand copies, gathered rows,
dz, routing counts, partial tiles and their counters, of the grouped and dense
products and of the GEMM paths behind linear_backward) stay valid when later
calls on the stream outgrow those workspaces."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def tmg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as t
    yield t
    t.check()


def ints(shape, seed):
    return torch.randint(-2, 3, shape, generator=torch.Generator().manual_seed(seed)).float().to(BF16).to(DEV)


def calls(tmg, scale):
    """One call for every workspace; larger with `scale`."""
    off = torch.tensor([0, 300 * scale, 1000 * scale], dtype=torch.int32, device=DEV)
    R = 1000 * scale
    x, W, d = ints((700 * scale, 265), 1)[:, 1:], ints((2, 264, 265), 2)[:, :, 1:], ints((R, 265), 3)[:, 1:]
    xa, Wa = ints((700, 264), 4), ints((2, 264 * scale, 264), 5)
    rows = torch.randint(0, 700, (R,), generator=torch.Generator().manual_seed(6)).int().to(DEV)
    logits = torch.randn(3000 * scale, 64, generator=torch.Generator().manual_seed(7)).to(DEV)
    dD, A, B = ints((640, 2048), 8), ints((640, 2560), 9), ints((2048, 2560), 10)
    sa, sb = ints((640 * scale, 2560), 11), ints((960 * scale, 2560), 12)
    cut = (1000, 5120, 4096) if scale == 1 else (1024, 8192, 8192)      # tiles of 224 and of 256 rows
    cutA, cutB = ints((cut[0], cut[2]), 13), ints((cut[1], cut[2]), 14)
    few, many = ints((16 * scale, 1024), 15), ints((1000 * scale, 1024), 16)
    deep = ints((3100, 264), 17)
    one = torch.tensor([0, 3100], dtype=torch.int32, device=DEV)
    return {"copies": lambda: [tmg.grouped_gemm(x[:R], W, off, rows=rows)],
            "gather": lambda: [tmg.grouped_gemm(xa, Wa, off, rows=rows)],
            "wgrad copies": lambda: [tmg.grouped_gemm_wgrad(d, x, off, rows=rows)],
            "wgrad cut": lambda: [tmg.grouped_gemm_wgrad(deep, deep, one)],
            "route": lambda: tmg.moe_route(logits, 6),
            "cut": lambda: [tmg.linear(cutA, cutB)],
            "backward": lambda: tmg.linear_backward(dD, A, B, preact=dD, activation="relu"),
            "stream-K": lambda: [tmg.gemm(sa, sb, path="tc_pair")],
            "layouts": lambda: [tmg.gemm(x, W[0], path="packed_tc")],
            "skinny": lambda: [tmg.gemm(few, many, path="skinny")]}


def test_graphs_survive_growing_workspaces(tmg, monkeypatch):
    torch.cuda.synchronize()
    tmg.shutdown()                                   # every workspace starts anew
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        small, large = calls(tmg, 1), calls(tmg, 4)
        s.synchronize()
        # the GEMM paths' stream-K partials grow with the tile width
        monkeypatch.setenv("TMG_TC_PAIR_SCHED", "sk")
        monkeypatch.setenv("TMG_TC_PAIR_BN", "128")
        want = {n: [t.clone() for t in f()] for n, f in small.items()}
        graphs = {}
        for n, f in small.items():
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                out = f()
            graphs[n] = g, out
        monkeypatch.setenv("TMG_TC_PAIR_BN", "256")
        for f in large.values():
            f()
        s.synchronize()
        # memory that a freed workspace would leave to others
        torch.cuda.empty_cache()
        others = [torch.full((n << 18,), 7, dtype=torch.int64, device=DEV) for n in (1, 1, 1, 2, 2, 4, 8, 16, 32)]
        for n, (g, out) in graphs.items():
            for t in out:
                t.zero_()
            for _ in range(2):
                g.replay()
            s.synchronize()
            for a, b in zip(out, want[n]):
                assert torch.equal(a, b), n
        assert all(bool((t == 7).all()) for t in others)
    tmg.check(s)


def test_first_call_inside_a_relaxed_capture(tmg):
    """The tile counters are made while the stream is captured; a call outside the graph
    comes before its first replay."""
    torch.cuda.synchronize()
    tmg.shutdown()
    A, B = ints((1000, 4096), 20), ints((5120, 4096), 21)
    want = tmg.linear(A, B)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        D, one = torch.empty_like(want), torch.empty_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s, capture_error_mode="relaxed"):
            tmg.linear(A, B, D)
        tmg.linear(A, B, one)
        for _ in range(2):
            D.zero_()
            g.replay()
        s.synchronize()
        assert torch.equal(one, want) and torch.equal(D, want)
        again = tmg.linear(A, B)
        s.synchronize()
    assert torch.equal(again, want)
    tmg.check(s)


def test_growth_inside_a_relaxed_capture(tmg):
    """A call inside the capture outgrows what one before it left, and one inside it
    again: the old buffers are kept, and the capture stays valid."""
    torch.cuda.synchronize()
    tmg.shutdown()
    sets = [(ints((n, 201), 30 + n)[:, 1:], ints((3 * n, 201), 31 + n)[:, 1:]) for n in (50, 300, 900)]
    want = [tmg.linear(A, B) for A, B in sets]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs = [torch.empty_like(w) for w in want]
        tmg.linear(*sets[0], outs[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s, capture_error_mode="relaxed"):
            for (A, B), D in zip(sets, outs):
                tmg.linear(A, B, D)
        for _ in range(2):
            for D in outs:
                D.zero_()
            g.replay()
        s.synchronize()
    assert all(torch.equal(D, w) for D, w in zip(outs, want))
    tmg.check(s)
