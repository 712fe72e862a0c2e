"""CPU: what the paged history's sources and its owner (runtime.PagedHistory) hold to
without a GPU."""
import os
import re

from jagged_pointwise_attention_hstu_b200 import build


def _source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_memory_that_another_kernel_may_write_is_read_by_ordinary_loads():
    """The kernels of the paged history start while the kernels before them still run, so none
    of what those may write (all memory but the handle's constant tables) is constant while
    they run, which is what the read-only path takes it for."""
    constant = {"time_lut", "thr32"}
    seen = set()
    for name in ("pages.cu", "pages.cuh", "pages_attn.cu"):
        text = _source(name)
        for arg in re.findall(r"__ldg\(([^;]*)", text):
            m = re.match(r"a\.(\w+)\b", arg)
            assert m and m.group(1) in constant, (name, arg[:60])
            seen.add(m.group(1))
        assert "__restrict__" not in text and "ld.global.nc" not in text, name
    assert seen <= constant


def test_a_warp_gives_up_a_wait_as_one():
    """Bounded waits are decided by the whole warp: lanes that look at the clock at different
    moments would part, and the rest wait for them in the next vote."""
    text = _source("pages_attn.cu")
    calls = re.findall(r"(?<!bool )\bwait_for\(", text)
    assert len(calls) == 1 and re.search(r"__all_sync\(0xffffffffu, wait_for\(", text)
    assert len(re.findall(r"(?<!bool )\bwait_by_all\(", text)) >= 4
