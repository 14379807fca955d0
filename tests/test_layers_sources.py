"""Source checks (no GPU) of the expert layer and the products with adapters."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_mma_atom_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", f.read()))


def between(text, start, end):
    return text.split(start, 1)[1].split(end, 1)[0]


def test_reads_before_the_kernels_own_wait_go_past_l1():
    """A kernel's own wait makes earlier kernels' writes visible to its loads; what it reads before that
    (adapters' numbers, scales, residual) it reads from L2."""
    read = between(source("lora.cuh"), "void read(const int32_t *adapters", "int next(")
    assert "__ldcg(adapters" in read and "adapters[" not in read
    rank = between(source("lora_rank.cu"), "lora_rank_kernel(const", "if (p.beside) grid_wait(); __syncwarp();")
    assert "__ldcg(p.adapters" in rank and "p.adapters[" not in rank and "p.scales[" not in rank
    first = between(source("lora_few.cu"), "void adapters_share(", "get_ranks(m0, rows);")
    assert "__ldcg(p.adapters" in first and "p.adapters[" not in first
    residual = between(source("moe_few.cu"), "void few_residual(", "void few_store(")
    assert residual.count("__ldcg(") == 2 and "= *reinterpret_cast" not in residual and "(r[j])" not in residual
    epilogue = source("lora_pair.cu").split("int local = 0; while (walk.next(tile, kb0, kb1, partial))")[1]
    assert 0 < epilogue.index("if (R || p.bias) grid_wait();") < epilogue.index("read(c_begin);")


def test_launch_rules_count_the_devices_sms():
    """No number of SMs, nor a multiple of one, stands in the kernels' sources."""
    for name in ("lora_few.cu", "lora_grad.cu", "lora_pair.cu", "lora_rank.cu", "lora_split.cu", "moe_few.cu", "few.cuh", "api_layers.cu"):
        numbers = [int(n) for n in re.findall(r"(?<![\w.])\d{3,}(?![\w.])", source(name))]
        assert not [n for n in numbers if n % 152 == 0 or n % 148 == 0], name
    assert "num_sms" in between(source("lora_few.cu"), "cudaError_t launch_lora_few_rank(", "}")
