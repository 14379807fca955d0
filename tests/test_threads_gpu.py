"""Host threads that share a stream: the kernels of one call (operand copy then
product, counts then plan) are not mixed with another call's."""
import threading

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


def jobs(tmg, seed, stream):
    """Calls that go through workspaces, on data of this seed."""
    g = torch.Generator().manual_seed(seed)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g).float().to(BF16).to(DEV)
    logits = torch.randn(3000 + 500 * seed, 64, generator=g).to(DEV)
    off = torch.tensor([0, 300, 300 + 100 * seed, 1200], dtype=torch.int32, device=DEV)
    rows = torch.randint(0, 700, (1200,), generator=g).int().to(DEV)
    A, B, d = ints(700, 201)[:, 1:], ints(3, 264, 201)[:, :, 1:], ints(1200, 265)[:, 1:]
    X, Wt = ints(500, 133)[:, 1:], ints(600, 133)[:, 1:]
    dD, P, A2, B2 = ints(300, 264), ints(300, 264), ints(300, 200), ints(264, 200)
    return [lambda: tmg.moe_route(logits, 6, stream=stream),
            lambda: [tmg.grouped_gemm(A, B, off, rows=rows, stream=stream)],
            lambda: [tmg.grouped_gemm_wgrad(d, A, off, rows=rows, stream=stream)],
            lambda: tmg.linear_backward(dD, A2, B2, preact=P, activation="relu", stream=stream),
            lambda: [tmg.gemm(X, Wt, path="packed_tc", stream=stream)]]


# 2 is cudaStreamPerThread: a stream, and workspaces, of each thread's own
@pytest.mark.parametrize("stream", [None, 2])
def test_threads_on_one_stream(tmg, stream):
    sets = [jobs(tmg, seed, stream) for seed in (1, 2, 3, 4)]
    torch.cuda.synchronize()
    want = [[list(job()) for job in js] for js in sets]
    torch.cuda.synchronize()
    bad, errors, start = [], [], threading.Barrier(len(sets))

    def work(i):
        try:
            start.wait()
            for _ in range(40):
                outs = [job() for job in sets[i]]
                if stream is not None:
                    torch.cuda.synchronize()
                for n, (got, ref) in enumerate(zip(outs, want[i])):
                    if not all(torch.equal(a, b) for a, b in zip(got, ref)):
                        bad.append((i, n))
        except Exception as x:      # noqa: BLE001 - reported below
            errors.append(repr(x))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert not bad, bad
    tmg.check()


def test_check_after_a_timeout_leaves_other_streams_alone(tmg):
    """A wait that ran out on one stream: the check resets the tile counters only when
    the calls under way on another have finished."""
    g = torch.Generator().manual_seed(9)
    A, B = (torch.randint(-2, 3, s, generator=g).float().to(BF16).to(DEV) for s in ((1000, 4096), (5120, 4096)))
    want = tmg.linear(A, B)
    busy, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        outs = [torch.empty_like(want) for _ in range(60)]
        tmg.linear(A, B, outs[0])
        busy.synchronize()
        for rounds in range(20):
            for D in outs:
                tmg.linear(A, B, D)
    tmg.debug_wait_timeout(1000, stream=other)
    with pytest.raises(tmg.TmgError, match="TIMEOUT"):
        tmg.check(other)
    with torch.cuda.stream(busy):
        outs.append(tmg.linear(A, B))
    busy.synchronize()
    assert all(torch.equal(D, want) for D in outs)
    tmg.check()
