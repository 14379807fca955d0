"""Calls on a stream other than the current one: results are not put into memory
that the current stream still reads, and inputs given up right after the call
keep theirs until its work is done."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
LONG = 400_000_000           # clock cycles of a kernel that only waits, 0.2 s


@pytest.fixture(scope="module")
def tmg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_mma_atom_gb300 as t
    yield t
    t.check()


def ints(shape, seed):
    return torch.randint(-2, 3, shape, generator=torch.Generator().manual_seed(seed)).float().to(BF16).to(DEV)


def calls(tmg):
    """Name -> (inputs, call(inputs, stream))."""
    T, E, k, H, F = 1024, 16, 4, 512, 384
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).to(DEV)
    r = tmg.moe_route(logits, k)
    x, W, y, d = ints((T, H), 2), ints((E, F, H), 3), ints((T * k, H), 4), ints((T * k, F), 5)
    return {
        "route": ([logits], lambda t, s: tmg.moe_route(t[0], k, stream=s)),
        "route_backward": ([logits, r.experts, r.weights], lambda t, s: [tmg.moe_route_backward(*t, stream=s)]),
        "combine": ([y, r.slots, r.weights], lambda t, s: [tmg.moe_combine(*t, stream=s)]),
        "combine_backward": ([x, y, r.slots, r.weights], lambda t, s: tmg.moe_combine_backward(*t, stream=s)),
        "grouped": ([x, W, r.offsets, r.rows], lambda t, s: [tmg.grouped_gemm(*t[:3], rows=t[3], stream=s)]),
        "wgrad": ([d, x, r.offsets, r.rows], lambda t, s: [tmg.grouped_gemm_wgrad(*t[:3], rows=t[3], stream=s)]),
        "linear": ([x, W[0].clone()], lambda t, s: [tmg.linear(*t, stream=s)]),
        "linear_backward": ([d[:T].clone(), x, W[0].clone()], lambda t, s: tmg.linear_backward(*t, stream=s)),
    }


NAMES = ["route", "route_backward", "combine", "combine_backward", "grouped", "wgrad", "linear", "linear_backward"]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_results_leave_the_current_streams_memory_alone(tmg, name, handle):
    inputs, call = calls(tmg)[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(inputs, None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.full_like(t, 3) for t in want]          # blocks of the results' sizes, to be given up
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    copies = [t.clone() for t in old]                    # queued behind the wait
    del old
    got = call(inputs, side.cuda_stream if handle else side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((c == 3).all()) for c in copies)
    tmg.check()


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_inputs_may_be_given_up_after_the_call(tmg, name, handle):
    inputs, call = calls(tmg)[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(inputs, None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    mine = [t.clone() for t in inputs]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    got = call(mine, side.cuda_stream if handle else side)
    shapes = [(t.shape, t.dtype) for t in mine]
    del mine
    junk = [torch.full(s, 5, dtype=d, device=DEV) for s, d in shapes for _ in range(2)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del junk
    tmg.check()
