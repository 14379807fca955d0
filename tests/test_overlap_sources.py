"""Source check (no GPU): kernels that start before their predecessor has ended
(launch.cuh) read nothing through non-coherent loads, which are for data that
nothing writes while the grid lives."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_mma_atom_gb300", "csrc")


def read(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_overlapped_kernels_use_plain_loads():
    names = sorted(n for n in os.listdir(CSRC) if "grid_wait()" in read(n))
    assert {"act_grad.cu", "pack3.cu", "route.cu", "split_kernel.cuh", "swap_kernel.cuh", "wgrad.cu"} <= set(names)
    for name in names + ["feed.cuh", "pieces.cuh", "staging.cuh", "act.cuh"]:
        text = read(name)
        assert "__ldg" not in text and "ld.global.nc" not in text, name
        assert not re.search(r"const\s+[\w:]+\s*\*\s*__restrict__", text), name


def test_kernels_settle_after_giving_up():
    """A kernel whose wait ran out leaves only when its loads have landed and its MMAs
    have run: those waits do not stop at the abort flag, and have a limit of their own."""
    flat = lambda name: re.sub(r"\s+", " ", read(name))
    body = flat("feed.cuh").split("void settle(")[1].split("constexpr")[0]
    assert "nullptr, kSiteDrain" in body and "1000000000ull" in body
    for name, loads, mmas in (("swap_kernel.cuh", "settle(full,", "settle(empty,"), ("wgrad.cu", "settle(full,", "settle(empty,"),
                              ("split_kernel.cuh", "settle(full,", "settle(done,")):
        text = flat(name)
        assert loads in text and mmas in text, name


def test_pieces_are_read_after_the_whole_warp_has_seen_the_arrival():
    """Between lane 0's acquire and the other lanes' reads stands a barrier of the warp:
    the shuffle that hands out the count orders no memory."""
    body = read("pieces.cuh").split("bool last_arrival(")[1].split("template")[0]
    before, after = body.split("atom.add.acq_rel.gpu")
    assert "__syncwarp()" in before and "__syncwarp()" in after.split("__shfl_sync")[0]
