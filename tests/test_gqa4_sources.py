"""What the sources of the 4-bit grouped-query and rotary kernels promise each
other."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "bit_kv_cache_nvfp4_gb300" / "csrc"


@pytest.mark.parametrize("name", ["kv4_gqa4.cu", "kv4_gqa4_attention.cu", "kv4_rotary.cu", "kv4_gqa_pages.cuh",
                                  "kv4_gqa_merge.cuh"])
def test_kernels_that_begin_early_read_nothing_as_read_only(name):
    """They are launched so that they may begin before the kernel before them has
    ended: each waits for it, and what that kernel may have written is not read
    through the path for data that nobody writes while a kernel runs."""
    code = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    for path in (r"__ldg\b", r"ld\.global\.nc", r"__restrict__"):
        assert not re.search(path, code), path
    kernels = code.split("__global__")[1:]
    assert bool(kernels) == (name != "kv4_gqa_pages.cuh")
    for body in kernels:
        before = body[:body.index("grid_dependency_wait()")]
        assert not re.search(r"\bload\(|\ba\.(cu|lens|scales|page_table|positions|inv_freq|dev_err)\b", before)


def test_a_warp_that_gave_up_frees_no_stage():
    """A stage of the rings is free when nothing is on its way to it any more, in a block
    that gave up too: who gave up its copies ends there and frees it no more; and the
    loading warp begins no copy behind the first stage that it did not get."""
    code = re.sub(r"//[^\n]*", "", (CSRC / "kv4_gqa4_attention.cu").read_text())
    assert len(re.findall(r"mbar_arrive\(smem_addr\(&sm\.(?:raw_)?empty\[", code)) == 2
    waits = re.findall(r"([^\n;{}]*)\bwait\(sm\.(?:raw_)?full\[[^;]*?\)\)\)([^;]*;[^;]*;)", code)
    assert len(waits) == len(re.findall(r"\bwait\(sm\.(?:raw_)?full\[", code)) == 2
    assert all("if (!__all_sync" in before and "break;" in after for before, after in waits)
    assert len(re.findall(r"stopped = __any_sync", code)) == len(re.findall(r"&& !stopped; ", code)) == 2
