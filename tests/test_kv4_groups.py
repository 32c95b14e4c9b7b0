"""The 4-bit cache's kernels: warps that give up a wait keep taking part in their group's barriers (checked in their source, as the
barriers themselves are in test_attention_groups.py)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "deepseek_sparse_mla_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_every_wait_of_the_few_row_kernel_is_bounded_and_its_groups_leave_together():
    text = source("kv4_attention.cu")
    assert not re.search(r"\b(named_bar|mbar_spin|mbar_wait)\s*\(", text)
    assert text.count("group_leave(bar, 128);") == 1
    # nothing but the loops' ends lies between a softmax warpgroup's last wait and its leaving
    tail = text[text.index("mbar_arrive(&q_empty[qb]);\n      }\n    }"):]
    assert tail.index("group_leave(bar, 128);") < tail.index("__syncthreads();")
    body = text[text.index("regs_inc<kRegsSoft>();"):text.index("group_leave(bar, 128);")]
    assert "return" not in re.sub(r"return (exists|e|r)\b[^\n]*", "", body)


def test_the_widening_warps_of_v_leave_their_group_before_the_common_one():
    text = source("paged_prompt.cu")
    widen = text[text.index("void pp_widen_v4("):text.index("template <bool k4, PaMods kModSet>")]
    assert "return" not in widen and widen.rstrip().endswith("group_leave(2, 128);\n}")
    assert set(re.findall(r"group_sync\((\d+), (\d+)\)", widen)) == {("2", "128")}


@pytest.mark.parametrize("name", ["kv4_attention.cu", "kv4_prompt.cu", "kv4_append.cu", "rope.cuh"])
def test_no_traps(name):
    assert not re.search(r"__trap|\bassert\s*\(", source(name))
