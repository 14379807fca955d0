"""The expert layer and the products with adapters beside other work: on a stream that is
not the current one, on several streams and from several host threads at once, captured
into graphs whose workspaces later calls outgrow, after kernels that write their inputs,
and through the bounds-checked build."""
import os
import threading

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


def rand(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(BF16).to(DEV)


def ids(M, L, run, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-1, L, (M // run + 1,), generator=g).repeat_interleave(run)[:M].int().to(DEV)


def calls(tmg, seed=0, scale=1):
    """Name -> (inputs, call(inputs, stream)): every kernel and every workspace of the three calls."""
    E, H, F, k, L = 16, 256 * scale, 128, 4, 5
    W1, W2 = rand((E, 2 * F, H), seed + 1, H ** -0.5), rand((E, H, F), seed + 2, F ** -0.5)
    out = {}
    for T in (1, 9, 40):
        x, g = rand((T, H), seed + 3 + T), rand((T, E), seed + 4 + T)
        out[f"moe {T}"] = ([x, g, W1, W2], lambda t, s: [tmg.moe_layer(*t, k, residual=t[0], stream=s)])
    for M, N, K, r, run in ((1, 264, 512, 16, 1), (33, 520, 1024 * scale, 16, 1), (64, 130, 257, 5, 2), (200, 384, 2048 * scale, 24, 30),
                            (900, 1032, 512, 16, 200), (2600 * scale, 1024, 1024, 16, 500), (300, 265, 203, 12, 50)):
        t = [rand((M, K), seed + M), rand((N, K), seed + N, K ** -0.5), rand((L, r, K), seed + 7, K ** -0.5),
             rand((L, N, r), seed + 8, r ** -0.5), ids(M, L, run, seed + M)]
        out[f"lora {M} {N} {K}"] = (t, lambda t, s: [tmg.lora_linear(*t, stream=s)])
        b = [rand((M, N), seed + 9)] + t + [rand((M, r), seed + 10)]
        out[f"grad {M} {N} {K}"] = (b, lambda t, s: tmg.lora_linear_backward(*t, stream=s))
    return out


@pytest.mark.parametrize("handle", [False, True])
def test_results_leave_the_current_streams_memory_alone(tmg, handle):
    for name, (inputs, call) in calls(tmg).items():
        side = torch.cuda.Stream()
        want = [t.clone() for t in call(inputs, None)]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        old = [torch.full_like(t, 3) for t in want]          # blocks of the results' sizes, to be given up
        torch.cuda.synchronize()
        torch.cuda._sleep(LONG // 8)
        copies = [t.clone() for t in old]                    # queued behind the wait
        del old
        got = call(inputs, side.cuda_stream if handle else side)
        torch.cuda.synchronize()
        assert all((c == 3).all() for c in copies), name
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    tmg.check()


def test_inputs_given_up_right_after_the_call(tmg):
    for name, (inputs, call) in calls(tmg).items():
        side = torch.cuda.Stream()
        want = [t.clone() for t in call(inputs, None)]
        mine = [t.clone() for t in inputs]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(LONG // 8)
        got = call(mine, side)
        sizes = [(t.shape, t.dtype) for t in mine]
        del mine
        junk = [torch.full(s, -1 if d is torch.int32 else float("nan"), dtype=d, device=DEV) for s, d in sizes]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        del junk
    tmg.check()


def test_streams_at_once(tmg):
    """Every call on four streams at the same time, over and over."""
    sets = [calls(tmg, 100 * i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in sets]
    want = [{n: [t.clone() for t in call(i, None)] for n, (i, call) in s.items()} for s in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [{} for _ in sets]
        for n in want[0]:
            for j, s in enumerate(sets):
                got[j][n] = s[n][1](s[n][0], streams[j])
        torch.cuda.synchronize()
        for j in range(len(sets)):
            for n in want[j]:
                assert all(torch.equal(a, b) for a, b in zip(got[j][n], want[j][n])), (j, n)
    tmg.check()


@pytest.mark.parametrize("stream", [None, 2])            # 2: cudaStreamPerThread
def test_threads_on_one_stream(tmg, stream):
    sets = [calls(tmg, 100 * i) for i in range(3)]
    want = [{n: [t.clone() for t in call(i, None)] for n, (i, call) in s.items()} for s in sets]
    torch.cuda.synchronize()
    bad, errors, start = [], [], threading.Barrier(len(sets))

    def work(j):
        try:
            start.wait()
            for _ in range(8):
                got = {n: call(i, stream) for n, (i, call) in sets[j].items()}
                if stream is not None:
                    torch.cuda.synchronize()
                bad.extend((j, n) for n in got if not all(torch.equal(a, b) for a, b in zip(got[n], want[j][n])))
        except Exception as x:      # noqa: BLE001 - reported below
            errors.append(repr(x))

    threads = [threading.Thread(target=work, args=(j,)) for j in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and not bad, (errors[:1], bad[:5])
    tmg.check()


def test_graphs_survive_growing_workspaces(tmg):
    torch.cuda.synchronize()
    tmg.shutdown()                                       # every workspace starts anew
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        small, large = calls(tmg), calls(tmg, scale=4)
        graphs = {}
        for n, (i, call) in small.items():
            want = [t.clone() for t in call(i, None)]
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                got = call(i, None)
            graphs[n] = (g, got, want)
        for i, call in large.values():
            call(i, None)
        s.synchronize()
        for n, (g, got, want) in graphs.items():
            for t in got:
                t.zero_()
            g.replay()
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), n
    tmg.check()


def test_graphs_on_two_streams_at_once(tmg):
    """The same calls captured on two streams and replayed at the same time."""
    streams, made = [torch.cuda.Stream() for _ in range(2)], []
    for j, s in enumerate(streams):
        with torch.cuda.stream(s):
            todo = calls(tmg, 50 * j)
            want = {n: [t.clone() for t in call(i, None)] for n, (i, call) in todo.items()}
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                got = {n: call(i, None) for n, (i, call) in todo.items()}
            made.append((g, got, want, todo))
    for _ in range(10):
        for s, (g, *_rest) in zip(streams, made):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, got, want, _ in made:
        for n in want:
            assert all(torch.equal(a, b) for a, b in zip(got[n], want[n])), n
    tmg.check()


def test_inputs_written_by_the_kernel_before(tmg):
    """Kernels start before the ones ahead of them have ended: every input written right before the call, by other
    kernels of the library too, and every result overwritten right after it."""
    for name, (inputs, call) in calls(tmg, 7).items():
        want = [t.clone() for t in call(inputs, None)]
        at = [torch.zeros_like(t) for t in inputs]
        torch.cuda.synchronize()
        for _ in range(20):
            for a, t in zip(at, inputs):
                a.zero_()
            tmg.linear(inputs[0], inputs[0])             # starts and ends like the call's own kernels
            for a, t in zip(at, inputs):
                a.copy_(t)
            got = [t.clone() for t in call(at, None)]
            again = call(at, None)
            for t in again:
                t.zero_()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
            assert not any(t.any() for t in again), name
    tmg.check()


def test_calls_that_read_each_others_results(tmg):
    """A row of calls, each reading what the last one wrote, equal to the same row with waits between."""
    L, r, E, k, F = 3, 8, 8, 2, 64
    for M in (1, 5, 40, 64, 100, 700):
        N = 256
        t = [rand((N, N), 1, N ** -0.5), rand((L, r, N), 2, N ** -0.5), rand((L, N, r), 3, r ** -0.5), ids(M, L, 7, 4)]
        W1, W2, router = rand((E, 2 * F, N), 5, N ** -0.5), rand((E, N, F), 6, F ** -0.5), rand((E, N), 7, N ** -0.5)
        u = torch.empty(M, r, dtype=BF16, device=DEV)

        def row(wait):
            x, out = rand((M, N), 8), []
            for _ in range(4):
                x = tmg.lora_linear(x, *t, residual=x, u=u)
                wait()
                g = tmg.linear(x, router)
                wait()
                x = tmg.moe_layer(x, g, W1, W2, k, residual=x)
                wait()
                d = tmg.lora_linear_backward(x, x, t[0], t[1], t[2], t[3], u)
                wait()
                x = (d[0].float() / 16).to(BF16)
                out += [x, *d[1:]]
            return out

        want = row(torch.cuda.synchronize)
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(row(lambda: None), want)), M
    tmg.check()


def test_debug_build_is_clean_and_equal(tmg):
    """Through the build whose kernels check every store and every access to partial sums."""
    from tiled_mma_atom_gb300 import _native, build
    build.build(debug_bounds=True)
    todo = calls(tmg, 3)
    want = {n: [t.clone() for t in call(i, None)] for n, (i, call) in todo.items()}
    tmg.check()
    _native.use_library(_native.DEBUG_LIB_PATH)
    try:
        assert _native.lib().tmg_debug_build() == 1
        got = {n: [t.clone() for t in call(i, None)] for n, (i, call) in todo.items()}
        tmg.check()
    finally:
        _native.use_library(os.path.join(_native.HERE, "libtmg.so"))
    for n in want:
        assert all(torch.equal(a, b) for a, b in zip(got[n], want[n])), n
