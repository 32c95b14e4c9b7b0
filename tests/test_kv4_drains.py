"""The 4-bit cache's kernels: a loader waits for all its copies in flight before its CTA ends, also where one of its waits ran out.
A wait cannot be made to run out on purpose on the GPU, so the loaders' bookkeeping is replayed here with the bounds that stand in
their source."""
import re

import pytest

from test_kv4_groups import source


def few_row_drain():
    """The drain's bound, with and without a wait that ran out, and whether the place that it was for is waited for."""
    text = source("kv4_attention.cu")
    loop = re.findall(r"for \(i -= 2; i >= 0 && i >= ([^;]+) - kRing; i -= 2\)", text)
    assert len(loop) == 1
    end = re.findall(r"const int end = ok \? (\w+) : (\w+);\s*(if \(!ok\) wait_warp\(&full\[st\], turn \^ 1,)?", text)
    return end[0] if loop[0] == "end" else (loop[0], loop[0], "")


def loader(first, ring, segments, stuck):
    """One of two loaders, tiles first, first + 2, ...; the product that reads tile `stuck` never ends.  Tiles that it issued, those
    that it waits for, and whether none of its waits ran out."""
    normal, failed, place = few_row_drain()
    i, i0, ok, issued = first, 0, True, []
    for n in segments:
        while ok and i - i0 < n:
            if i >= ring and i - ring >= stuck:
                ok = False
                break
            issued.append(i)
            i += 2
        i0 += n
        if not ok:
            break
    bound = {"i0": i0, "i": i}[normal if ok else failed] - ring
    waited = {t for t in issued if t >= bound}
    return issued, waited | ({i - ring} if not ok and place else set()), ok


@pytest.mark.parametrize("ring", [4, 5, 6])
@pytest.mark.parametrize("segments", [[1], [3, 1, 1, 2], [40], [1] * 9, [7, 30, 2], []])
def test_few_row_loaders_wait_for_their_last_copies(ring, segments):
    none = 10 ** 6
    for stuck in [*range(sum(segments)), none]:
        both = [loader(first, ring, segments, stuck) for first in (0, 1)]
        issued = {t for tiles, _, _ in both for t in tiles}
        last = {t for t in issued if t + ring not in issued}   # nothing has been loaded over them
        for tiles, waited, ok in both:
            assert waited <= last, "a wait for what has been loaded over"
            assert ok or stuck != none
            if stuck == none:
                assert waited == last & set(tiles)
        waited = both[0][1] | both[1][1]
        assert waited >= {t for t in issued if t >= stuck}, (stuck, both)   # those before it have been used


def test_the_prompt_kernel_waits_for_every_tile_that_it_copies():
    """Its loader notes a tile of K or V as it asks for it, whatever ends the loop after that, and the last of those in each of the two
    places is waited for."""
    text = source("paged_prompt.cu")
    after = re.findall(r"\n\s*copy_raw\((?:[^;]*)\);\s*([^;]+);", text)
    assert sorted(after) == ["k_tiles = i + 1", "v_tiles = j + 1"]
    drain = text[text.index("auto landed = "):]
    assert re.search(r"landed\(rawk_full, k_tiles\);\s*landed\(rawv_full, v_tiles\);", drain)
    parity = re.search(r"if \(tiles > rb\) wait_warp\(&full\[rb\], (.+) & 1, err", drain).group(1).replace("/", "//")
    places = int(re.search(r"kRawStages = (\d+);", text).group(1))
    for tiles in range(12):
        for rb in range(places):
            uses = len(range(rb, tiles, places))
            if uses:
                assert eval(parity, {}, {"tiles": tiles, "rb": rb, "kRawStages": places}) & 1 == (uses - 1) & 1
