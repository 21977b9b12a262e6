"""What the sources of the 8-bit grouped-query kernels promise each other."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "bit_kv_cache_nvfp4_gb300" / "csrc"


@pytest.mark.parametrize("name", ["kv4_gqa8.cu", "kv4_gqa8_attention.cu", "kv4_gqa8_device.cuh"])
def test_kernels_that_begin_early_read_nothing_as_read_only(name):
    """They are launched so that they may begin before the kernel before them
    has ended: each waits for it, and what that kernel may have written is not
    read through the path for data that nobody writes while a kernel runs."""
    text = (CSRC / name).read_text()
    code = re.sub(r"//[^\n]*", "", text)
    for path in (r"__ldg\b", r"ld\.global\.nc", r"__restrict__"):
        assert not re.search(path, code), path
    kernels = code.split("__global__")[1:]
    assert bool(kernels) == name.endswith(".cu")
    for body in kernels:
        before = body[:body.index("grid_dependency_wait()")]
        assert not re.search(r"\bload\(|\ba\.(cu|lens|scales|page_table|dev_err)\b", before)


@pytest.mark.parametrize("name,kernels", [("kv4_gqa8_attention.cu", 2), ("kv4_gqa4_attention.cu", 1)])
def test_queued_products_end_before_a_block_does(name, kernels):
    """Whoever gives up a wait may do so behind the last product's issue, so whether a
    block has given up is looked at behind the barrier that all its waits come before."""
    code = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    ends = re.findall(r"__syncthreads\(\);\s*if \(warp == 1\) \{\s*if \(__any_sync\(0xFFFFFFFFu, \*dead != 0\)\) \{\s*"
                      r"if \(elect_one\(\)\) mma_commit\(smem_addr\(&sm\.never\)\);\s*__syncwarp\(\);\s*"
                      r"mbar_wait_bounded\(smem_addr\(&sm\.never\)[^}]*\}\s*tmem_dealloc", code)
    assert len(ends) == kernels == code.count("mma_commit(smem_addr(&sm.never))") == code.count("tmem_dealloc(")
