"""Which kernel and schedule the products take (as TMG_LOG reports them), so that a
change of a rule cannot leave a branch without its tests."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def log_of(code):
    """The library's log of a program that has torch, tmg and normal(rows, cols)."""
    head = ("import __graft_entry__ as g\ng.build()\nimport torch\nimport tiled_mma_atom_gb300 as tmg\n"
            "normal = lambda m, n: torch.randn(m, n, device='cuda').to(torch.bfloat16)\n")
    r = subprocess.run([sys.executable, "-c", head + code + "\ntmg.check()\n"], cwd=ROOT, capture_output=True, text=True,
                       env=dict(os.environ, TMG_LOG="1"), timeout=300)
    assert r.returncode == 0, r.stderr
    return [line for line in r.stderr.splitlines() if line.startswith("tmg: ")]


def test_dense_tiles_are_cut_where_the_estimate_says():
    """1000 x 5120 x 4096: 100 tiles of 224 rows over 76 pairs, 24 of them cut over
    three pairs each; contractions of 3000 are too short for a cut, and the log, the
    kernel and the choice of the width agree on that."""
    lines = log_of("for m, n, k in ((1000, 5120, 4096), (2489, 5648, 3000)):\n"
                   "    tmg.linear(normal(m, k), normal(n, k))")
    assert len(lines) == 2 and all("swap_kernel" in line for line in lines)
    assert "24 tiles cut over 72 pairs" in lines[0]
    assert "cut" not in lines[1]


def test_gradient_copies_no_operand_for_less_than_256_rows():
    """200 x 4096 x 20480: 80 tiles would fill the CTA pairs, but the GEMM reads
    MN-major operands in place from 256 rows on only."""
    lines = log_of("tmg.linear_backward(normal(200, 4096), normal(200, 20480), normal(4096, 20480))")
    assert "dense: 200 rows" in lines[0]
    assert not any("200x20480x4096" in line for line in lines)


GRADIENT = """
def ints(m, n, seed):
    return torch.randint(-2, 3, (m, n), generator=torch.Generator('cuda').manual_seed(seed), device='cuda').to(torch.bfloat16)
M, N, K = {size}
dD, A, B, pre = ints(M, N, 1), ints(M, K, 2), ints(N, K, 3), ints(M, N, 4)
dA, dB, db = tmg.linear_backward(dD, A, B, preact=pre, activation="relu")
tmg.check()
dz = torch.where(pre > 0, dD, 0).double()
assert torch.equal(dA, (dz @ B.double()).to(torch.bfloat16)), "dA"
assert torch.equal(dB, (dz.T @ A.double()).to(torch.bfloat16)), "dB"
assert torch.equal(db.double(), dz.sum(0)), "dbias"
"""


# every branch of the gradient's choice: integers, so all three results are exact
@pytest.mark.parametrize("size,dA,dB", [
    ((1024, 4096, 4096), "product", "gemm"),         # dA's tiles do not fill the pairs
    ((8191, 4096, 4096), "gemm", "wgrad"),           # the longest side is the rows; dz in chunks of 128 rows
    ((2048, 4096, 4096), "gemm", "gemm"),
    ((2048, 8192, 4096), "product", "gemm"),         # a contraction of more than 4096 columns
    ((2560, 2048, 2560), "gemm", "gemm stream-K"),
    ((2048, 4104, 4104), "product", "wgrad"),        # rows that begin inside a sector
    ((48, 4096, 8192), "product", "wgrad"),          # less than 64 rows
    ((255, 4096, 20480), "product", "gemm"),         # less than 256 rows
])
def test_every_branch_of_the_dense_gradient_is_exact(size, dA, dB):
    M, N, K = size
    lines = log_of(GRADIENT.format(size=size))
    gemm = [line for line in lines if "tc2_gemm_kernel" in line and "read in place" in line]
    taken = {"product": any(f"dense: {M} rows, N={K} K={N} " in line for line in lines),
             "gemm": any(f"bf16 {M}x{K}x{N} " in line for line in gemm)}
    assert taken[dA], lines
    taken = {"wgrad": any(f"weight gradient: {M} rows, N={N} K={K} " in line for line in lines),
             "gemm": any(f"bf16 {N}x{K}x{M} " in line for line in gemm),
             "gemm stream-K": any(f"bf16 {N}x{K}x{M} " in line and "+ 0 stream-K" not in line for line in gemm)}
    assert taken[dB], lines
