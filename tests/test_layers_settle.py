"""After a wait ran out, a kernel of few rows leaves shared memory only when its copies have
landed (no GPU): the ring's barriers modelled on the host, with the kernels' own code for
the two producers' last waits, for every number of stages that each had issued."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_mma_atom_gb300", "csrc")

MODEL = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>
#define __device__
#define __noinline__
#define __forceinline__
#define __syncwarp()
constexpr int kFwMaxStages = 12, kSiteDrain = 5, WEIGHTS = 16384;
struct ErrCtx { uint32_t *word; uint64_t budget_ns; };
struct FewShape { int tp, stages, stage_bytes, ring_bytes, tmem_cols; };
// a barrier of one arrival and bytes; a copy under way to it
struct Bar { int phase = 0, pending = 1; long tx = 0; };
struct Copy { int bar; long bytes; };
struct FewRing { uint64_t full[kFwMaxStages]; int issued[2]; };
static Bar bars[kFwMaxStages];
static std::vector<Copy> flying;
static FewRing ring;
static int lost;
static void settled(Bar &b) { if (b.pending == 0 && b.tx == 0) { ++b.phase; b.pending = 1; } }
static void land(size_t i) { Copy c = flying[i]; flying.erase(flying.begin() + i); bars[c.bar].tx -= c.bytes; settled(bars[c.bar]); }
static void mbar_arrive_expect_tx_w(uint64_t *bar, uint32_t bytes)
{
    Bar &b = bars[bar - ring.full];
    if (b.pending != 1) { std::printf("a second arrival in a phase\n"); std::exit(1); }
    b.pending = 0; b.tx += bytes; settled(b);
}
static bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, const ErrCtx &, volatile int *, int)
{
    Bar &b = bars[bar - ring.full];
    for (;;) {
        if (uint32_t(b.phase & 1) != parity) return true;
        if (flying.empty()) { ++lost; return false; }          // a second is over: all copies have landed
        land(std::rand() % flying.size());
    }
}
SETTLE
ROWS
int main()
{
    const long tp = 32, rows = tp * 128;
    for (int stages = 2; stages <= kFwMaxStages; ++stages)
        for (int done = 0; done <= 2 * stages + 1; ++done)              // stages that the MMAs have read
            for (int w = done; w <= done + stages; ++w)                 // issued by the weights' producer
                for (int r = done; r <= done + stages; ++r)             // and by the rows'
                    for (int seed = 0; seed < 5; ++seed) {
                        std::srand(seed);
                        for (int s = 0; s < kFwMaxStages; ++s) bars[s] = Bar();
                        flying.clear(); lost = 0;
                        for (int u = 0; u < (w > r ? w : r); ++u) {
                            const int s = u % stages;
                            if (u < w) { mbar_arrive_expect_tx_w(&ring.full[s], WEIGHTS + rows); flying.push_back({s, WEIGHTS}); }
                            if (u < r) flying.push_back({s, rows});
                            if (u < done) while (bars[s].phase <= u / stages) land(flying.size() - 1);
                        }
                        for (int i = std::rand() % 3; i > 0 && !flying.empty(); --i) land(std::rand() % flying.size());
                        FewShape p{(int)tp, stages, 0, 0, 0};
                        ErrCtx err{nullptr, 1};
                        ring.issued[0] = w;
                        ring.issued[1] = r;
                        const int n = few_announce(p, ring);
                        settle(ring.full, p.stages, n % p.stages, n / p.stages & 1, n, err.word, err.budget_ns);
                        if (!flying.empty() || (lost && r >= w)) {
                            std::printf("%d stages, %d read, %d and %d issued: %zu copies under way, %d waits ran out\n", stages, done, w, r, flying.size(), lost);
                            return 1;
                        }
                    }
    return 0;
}
"""


def function(name, head):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return head + text.split(head, 1)[1].split("\n}\n", 1)[0] + "\n}\n"


def test_both_producers_copies_have_landed(tmp_path):
    code = MODEL.replace("SETTLE", function("feed.cuh", "static __device__ __noinline__ void settle("))
    code = code.replace("ROWS", function("few.cuh", "__device__ __forceinline__ int few_announce("))
    src, exe = tmp_path / "settle.cpp", tmp_path / "settle"
    src.write_text(code)
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-o", str(exe), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_both_kernels_of_few_rows_wait_for_the_rows_copies():
    last = "const int n = few_announce({0}, sm); settle(sm.full, {0}.stages, n % {0}.stages, n / {0}.stages & 1, n, err.word, err.budget_ns);"
    for name, call in (("few.cuh", last.format("p")), ("moe_few.cu", last.format("p.shape"))):
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", f.read()))
        before, after = text.split(call)
        assert "sm.issued[warp / 2] = issued;" in before
        # between the two: a barrier of all warps
        assert re.search(r"cluster_sync\(\);|__syncthreads\(\);", before.split("sm.issued[warp / 2] = issued;")[1]), name
