"""The expert layer and the products with adapters where the other tests do not go: the pair
kernel's cut tiles, forward and backward, also on several streams and threads, in graphs
and through the bounds-checked build; the layer by groups there; operands of the gradients
that are views; factors and weights that start at any element."""
import pytest
import torch

from tests import test_layers_streams_gpu as base
from tests.test_grouped_schedule_gpu import log_of
from tests.test_layers_gpu import (BF16, DEV, F32, check_grads, check_layer, check_lora, ids_of, lora_inputs, moe_inputs, normal)
from tests.test_layers_streams_gpu import ids, rand

pytestmark = pytest.mark.gpu

# rows, N, K, rank: products whose last wave of tiles is cut, and in how many pieces
CUT = [(520, 2056, 6000, 16, "33 tiles cut over 66 pairs"), (300, 3500, 5000, 24, "38 tiles cut over 76 pairs"),
       (260, 9900, 5000, 8, "14 tiles cut over 70 pairs")]
# the same of the input's gradient, N its contraction
CUT_BACK = [(300, 6000, 5200, 16, "6 tiles cut over 48 pairs"), (2300, 4104, 2056, 40, "5 tiles cut over 40 pairs")]


@pytest.fixture(scope="module")
def tmg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as t
    yield t
    t.check()


def test_these_tiles_are_cut():
    """By the library's log."""
    lines = log_of("of = lambda m: torch.zeros(m, dtype=torch.int32, device='cuda')\n"
                   f"for m, n, k, r, _ in {CUT!r}:\n"
                   "    tmg.lora_linear(normal(m, k), normal(n, k), normal(r, k)[None], normal(n, r)[None], of(m))\n"
                   f"for m, n, k, r, _ in {CUT_BACK!r}:\n"
                   "    tmg.lora_linear_backward(normal(m, n), normal(m, k), normal(n, k), normal(r, k)[None], normal(n, r)[None], of(m), normal(m, r))")
    lines = [line for line in lines if "lora_pair_kernel" in line]
    assert len(lines) == len(CUT) + len(CUT_BACK)
    for line, (*_, cut) in zip(lines, CUT + CUT_BACK):
        assert line.endswith(cut), line


@pytest.mark.parametrize("kind", ["runs", "each", "outside"])
@pytest.mark.parametrize("M,N,K,r,_", CUT)
def test_cut_tiles(tmg, M, N, K, r, _, kind):
    """Adapters' blocks in a tile's last piece; bias, and a residual that is D, added by the last pair."""
    t, of = lora_inputs(M, N, K, r, 7, 400), ids_of(kind, M, 7, 401)
    bias, res = normal(N, 402, dtype=F32), normal((M, N), 403)
    D, _ = check_lora(tmg, t, of, bias=bias, residual=res)
    here = res.clone()
    tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], of, here, scales=t["scales"], bias=bias, residual=here)
    assert torch.equal(here, D)
    for _ in range(5):
        assert torch.equal(tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], of, scales=t["scales"], bias=bias, residual=res), D)


@pytest.mark.parametrize("kind", ["runs", "outside"])
@pytest.mark.parametrize("M,N,K,r,_", CUT_BACK)
def test_cut_tiles_of_the_inputs_gradient(tmg, M, N, K, r, _, kind):
    t, of = lora_inputs(M, N, K, r, 5, 410), ids_of(kind, M, 5, 411)
    check_grads(tmg, t, of, normal((M, N), 412), normal((M, r), 413))


def test_cut_tiles_keep_requests_apart(tmg):
    """Infinities of an adapter reach no row that has another one, nor one without."""
    M, N, K, r, _ = CUT[0]
    t, of = lora_inputs(M, N, K, r, 4, 420), ids_of("each", M, 3, 421)
    of[77] = 3
    want = tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], of)
    t["A"][3, 1, K - 1], t["B"][3] = float("inf"), float("nan")
    got = tmg.lora_linear(t["x"], t["W"], t["A"], t["B"], of)
    tmg.check()
    others = torch.arange(M, device=DEV) != 77
    assert torch.equal(got[others], want[others]) and not got[77].isfinite().any()


# ------------------------------------------------- beside other work

def more_calls(tmg, seed=0, scale=1):
    """Name -> (inputs, call(inputs, stream)), as test_layers_streams_gpu's: cut tiles, and the layer by groups."""
    out = {}
    for T, H in ((100 * scale, 256), (9, 130), (70, 264)):
        E, F, k = 16, 128, 4
        t = [rand((T, H), seed + T), rand((T, E), seed + 1), rand((E, 2 * F, H), seed + 2, H ** -0.5), rand((E, H, F), seed + 3, F ** -0.5)]
        out[f"moe {T} {H}"] = (t, lambda t, s: [tmg.moe_layer(*t, 4, residual=t[0], stream=s)])
    L = 5
    for M, N, K, r, _ in CUT[:2]:
        t = [rand((M, K), seed + M), rand((N, K), seed + N, K ** -0.5), rand((L, r, K), seed + 7, K ** -0.5),
             rand((L, N, r), seed + 8, r ** -0.5), ids(M, L, 40, seed + M), rand((M, N), seed + 9)]
        out[f"lora {M} {N} {K}"] = (t, lambda t, s: [tmg.lora_linear(*t[:5], residual=t[5], stream=s)])
    M, N, K, r, _ = CUT_BACK[0]
    t = [rand((M, N), seed + 9), rand((M, K), seed + M), rand((N, K), seed + N, K ** -0.5), rand((L, r, K), seed + 7, K ** -0.5),
         rand((L, N, r), seed + 8, r ** -0.5), ids(M, L, 40, seed + M), rand((M, r), seed + 10)]
    out[f"grad {M} {N} {K}"] = (t, lambda t, s: tmg.lora_linear_backward(*t, stream=s))
    return out


@pytest.mark.parametrize("test,args", [
    (base.test_results_leave_the_current_streams_memory_alone, (False,)), (base.test_inputs_given_up_right_after_the_call, ()),
    (base.test_streams_at_once, ()), (base.test_threads_on_one_stream, (None,)), (base.test_threads_on_one_stream, (2,)),
    (base.test_graphs_survive_growing_workspaces, ()), (base.test_graphs_on_two_streams_at_once, ()),
    (base.test_inputs_written_by_the_kernel_before, ()), (base.test_debug_build_is_clean_and_equal, ())],
    ids=lambda v: v.__name__[5:] if callable(v) else "-".join(map(str, v)) or "all")
def test_beside_other_work(tmg, monkeypatch, test, args):
    monkeypatch.setattr(base, "calls", more_calls)
    test(tmg, *args)


# ------------------------------------------------- views and odd addresses

@pytest.mark.parametrize("M,r", [(3, 16), (60, 12), (200, 16), (400, 64)])
@pytest.mark.parametrize("off", [0, 8, 3])
def test_gradients_of_views(tmg, M, r, off):
    """dD, x and W as views of wider matrices, on 16-byte borders and off them."""
    N, K = 264, 200
    t = lora_inputs(M, N, K, r, 4, 430)
    t["x"] = normal((M, K + 56), 431)[:, off:off + K]
    t["W"] = normal((N, K + 24), 432, 0.1)[:, off:off + K]
    dD = normal((M, N + 40), 433)[:, off:off + N]
    check_grads(tmg, t, ids_of("runs", M, 4, 434), dD, normal((M, r), 435))
    check_grads(tmg, t, ids_of("each", M, 4, 434), dD, normal((M, r), 435), scaled=False)


def test_gradients_of_broadcast_rows(tmg):
    """A row stride of zero in dD and x."""
    M, N, K, r = 130, 136, 72, 8
    t, of, u = lora_inputs(M, N, K, r, 3, 440), ids_of("runs", M, 3, 441), normal((M, r), 442)
    t["x"] = normal((1, K), 443).expand(M, K)
    check_grads(tmg, t, of, normal((1, N), 444).expand(M, N), u)
    check_lora(tmg, t, of)


def shifted(t, by):
    """The same values, contiguous, `by` elements after a 16-byte border."""
    room = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    room[by:] = t.reshape(-1)
    return room[by:].view(t.shape)


@pytest.mark.parametrize("by", [1, 4, 8])
@pytest.mark.parametrize("M,r", [(1, 16), (5, 16), (64, 64), (150, 16), (700, 24)])
def test_factors_at_any_element(tmg, M, r, by):
    t = lora_inputs(M, 264, 328, r, 4, 450)
    of, dD = ids_of("runs", M, 4, 451), normal((M, 264), 452)
    for names in (("A",), ("B",), ("A", "B"), ("x", "W", "A", "B")):
        s = {k: shifted(v, by) if k in names else v for k, v in t.items()}
        _, u = check_lora(tmg, s, of, name=str(names))
        check_grads(tmg, s, of, shifted(dD, by), shifted(u, by), name=str(names))
        got = torch.full((M * r + by + 3,), 7.0, dtype=BF16, device=DEV)
        tmg.lora_linear(s["x"], s["W"], s["A"], s["B"], of, scales=s["scales"], u=got[by:by + M * r].view(M, r))
        assert torch.equal(got[by:by + M * r].view(M, r), u) and (got[:by] == 7).all() and (got[by + M * r:] == 7).all()


@pytest.mark.parametrize("by", [1, 4, 8])
@pytest.mark.parametrize("T", [1, 13, 40, 90])
def test_weights_of_experts_at_any_element(tmg, T, by):
    x, logits, W1, W2, res = moe_inputs(T, 12, 136, 72, 460)
    for names in ("1", "2", "12", "x12r"):
        check_layer(tmg, shifted(x, by) if "x" in names else x, shifted(logits, by) if "r" in names else logits,
                    shifted(W1, by) if "1" in names else W1, shifted(W2, by) if "2" in names else W2, 3,
                    residual=shifted(res, by) if "r" in names else res, name=names)


@pytest.mark.parametrize("M", [40, 130, 700])
def test_rows_that_overlap(tmg, M):
    """Inputs whose row stride is less than a row: any other one is read, so are these."""
    N, K, r = 136, 72, 8
    t, of, u = lora_inputs(M, N, K, r, 3, 470), ids_of("runs", M, 3, 471), normal((M, r), 472)
    t["x"] = normal((M * 8 + K,), 473).as_strided((M, K), (8, 1))
    t["W"] = normal((N * 64 + K,), 474, 0.1).as_strided((N, K), (64, 1))
    check_lora(tmg, t, of, residual=normal((M * 8 + N,), 475).as_strided((M, N), (8, 1)))
    check_grads(tmg, t, of, normal((M * 8 + N,), 476).as_strided((M, N), (8, 1)), u)
    _, logits, W1, W2, _ = moe_inputs(M, 8, K, 40, 477)
    check_layer(tmg, t["x"], logits, W1, W2, 2)
    offsets = torch.tensor([0, M // 3, M], dtype=torch.int32, device=DEV)
    ints = lambda rows, cols, ld, seed: normal((rows * ld + cols,), seed).round().as_strided((rows, cols), (ld, 1))       # exact sums
    a, b = ints(M, K, 8, 478), ints(N, K, 64, 479)
    assert torch.equal(tmg.linear(a, b), (a.double() @ b.double().T).to(BF16))
    B = normal((2, N, K), 480).round()
    want = torch.cat([a[:M // 3].double() @ B[0].double().T, a[M // 3:].double() @ B[1].double().T]).to(BF16)
    assert torch.equal(tmg.grouped_gemm(a, B, offsets), want)
    tmg.check()
