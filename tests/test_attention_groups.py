"""Warps of the dense attention kernels that share scratch or meet at a barrier, checked on the CPU from the kernels' source:
the GPU can only show that a race did not happen."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deepseek_sparse_mla_gb300", "csrc")
BARRIER = r"\b\w+_sync\(bar, 128\)"


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_segments_sums_are_read_before_the_next_segments_maxima_replace_them():
    """One warp of a softmax warpgroup reads what all four left in wmax.  Both ways on from there (this warpgroup writes the
    segment's outputs, or the other one does) pass a barrier of the warpgroup before any warp writes wmax again."""
    text = source("paged_attention.cu")
    read = re.search(r"\(wmax\[wg\]\[0\]\[lane\] \+ wmax\[wg\]\[1\]\[lane\]\)", text)
    other = re.search(r"if \(\(seg & 1\) != wg\) \{(.*?)continue;\s*\}", text[read.end():], re.S)
    assert re.search(BARRIER, other.group(1)), "the warpgroup that does not write the outputs goes on without a barrier"
    writer = text[read.end() + other.end():]
    writer = writer[:writer.index("a.out[")]
    assert re.search(BARRIER, writer) and "wmax" not in writer[:re.search(BARRIER, writer).start()]
    before = text[:read.start()]                            # and the sums are complete when they are read
    assert before.rindex("wmax[wg][quarter][c] = v") < [m.start() for m in re.finditer(BARRIER, before)][-1]
