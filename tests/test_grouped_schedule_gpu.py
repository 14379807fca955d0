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
