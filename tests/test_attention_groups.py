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


def run_group(scripts):
    """Warps that meet at one counting barrier: a script is the votes (0 or 31 threads) of the barriers a warp takes part in
    before it is done or gives up; then it votes with all 32 until every warp does.  Returns the phase each one left at."""
    at, left, results = [0] * len(scripts), [None] * len(scripts), [[] for _ in scripts]
    for phase in range(1 + max(map(len, scripts))):
        votes = [s[i] if i < len(s) else 32 for s, i in zip(scripts, at)]
        count = sum(votes)
        for w, s in enumerate(scripts):
            if at[w] < len(s):
                results[w].append((count & 31) != 0)
                at[w] += 1
            elif count == 32 * len(scripts):
                left[w] = phase
    return left, results


def test_a_group_leaves_together_wherever_its_warps_give_up():
    """Every place to give up for every warp, with every vote: all leave at the same barrier, none waits for one that has
    left, and a vote counts if and only if a warp that goes on has cast it."""
    import itertools
    for warps, length in ((4, 3), (8, 2)):
        for ends in itertools.product(range(length + 1), repeat=warps):
            for yes in (range(2 ** length) if warps == 4 else (0, 1, 3)):
                vote = [31 * (yes >> i & 1) for i in range(length)]
                scripts = [vote[:e] if w % 2 else [v * (w == 0) for v in vote[:e]] for w, e in enumerate(ends)]
                left, results = run_group(scripts)
                assert None not in left and len(set(left)) == 1 and left[0] == max(ends)
                for got in results:
                    for i, r in enumerate(got):
                        assert r == any(len(s) > i and s[i] for s in scripts)


def test_groups_have_no_barrier_that_a_warp_that_gave_up_would_miss():
    for name, leave in (("paged_attention.cu", "group_leave(bar, 128);"), ("paged_prompt.cu", "group_leave(1, 256);")):
        text = source(name)
        assert "named_bar" not in text and text.count(leave) == 1
        # nothing but the next role (or the kernel's end) follows: every way out of the walk over the segments comes here
        rest = text[text.index(leave) + len(leave):].split()
        assert rest[0] == "}" and rest[1] in ("else", "tc_fence_before();")
        # and a warp's lanes agree on giving up
        assert not re.search(r"\bmbar_(spin|wait)\(", text)


def test_the_sums_of_the_prompt_kernels_split_stay_in_32_bits():
    """Its sums over the requests, for the largest batches that the host lets through, whatever the row offsets say: a thread's
    share of the entries is held at one more than requests without shared rows can have, and more of them are refused."""
    requests, pairs = 4096, 2 ** 30                        # DSA_MAX_REQUESTS; rows * heads, as checked by the host
    most = pairs // 256 + requests
    threads, entries = 640, pairs // 256                   # of one request that names every row
    alternating = requests // 2 * entries                  # every other request does
    assert alternating > 2 ** 31                           # what an unchecked sum would be
    assert threads * (most + 1) < 2 ** 32
    text = source("paged_prompt.cu")
    assert "min(sum + pp_entries(a, pa_shape(a, b, bits)), most_entries + 1)" in text
    assert re.search(r"entry_end\[B - 1\] > most_entries\) \{\s*entry_end\[B - 1\] = 0;", text)
    api = source("dsa_api.cu")
    assert "num_rows * q_heads > INT32_MAX / 2" in api and "num_rows * group / 256 + batch->num_requests" in api
