"""Which operands the tensor maps read where they stand (no GPU): the rule itself, compiled
for the host."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "product.h"
#include <cstdio>
#include <cstdlib>
int main(int argc, char **argv)
{
    for (int i = 1; i + 5 < argc; i += 6) {
        long long v[6];
        for (int j = 0; j < 6; ++j) v[j] = std::atoll(argv[i + j]);
        std::printf("%d", tmg::rows_in_place(reinterpret_cast<void *>(v[0]), v[1], v[2], v[3], v[4], int(v[5])));
    }
}
"""


def in_place(tmp_path, *cases):
    """cases: (address, rows, row stride, columns, column stride, bytes of an element)."""
    from tiled_mma_atom_gb300 import build
    src, exe = tmp_path / "rows.cu", tmp_path / "rows"
    src.write_text(PROGRAM)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, "-o", str(exe), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)] + [str(v) for c in cases for v in c], capture_output=True, text=True).stdout
    return [d == "1" for d in out]


def test_rows_that_overlap_are_copied(tmp_path):
    """A tensor map's rows lie one after another: a row stride below the row's own extent is not one of its forms."""
    assert in_place(tmp_path, (4096, 130, 8, 72, 1, 2), (4096, 130, 64, 72, 1, 2), (4096, 130, 72, 72, 1, 2), (4096, 130, 80, 72, 1, 2),
                    (4096, 1, 8, 72, 1, 2), (4096, 5, 16, 32, 1, 1), (4096, 5, 32, 32, 1, 1)) == [False, False, True, True, True, False, True]


def test_rows_off_the_borders_are_copied(tmp_path):
    assert in_place(tmp_path, (4098, 4, 72, 72, 1, 2), (4096, 4, 76, 72, 1, 2), (4096, 4, 0, 72, 1, 2), (4096, 4, 72, 72, 2, 2),
                    (4096, 4, 72, 0, 1, 2), (4096, 0, 72, 72, 1, 2)) == [False] * 6
