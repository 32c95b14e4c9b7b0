"""The dense layer's oracle against brute force and closed forms (CPU)."""
import math

import numpy as np
import pytest

from dense_cases import DenseCase
from oracle import dense_oracle as d
from oracle import dsa_oracle as o


def test_block_scale_is_the_smallest_power_of_two_that_holds_the_block():
    rng = np.random.default_rng(0)
    for x in list(rng.standard_normal(50) * 10.0 ** rng.uniform(-20, 20, 50)) + [448.0, 448.0001, 447.999, 224.0, 1.75 * 2.0 ** 30]:
        s = d.block_scale([x, x / 3])
        assert math.frexp(s)[0] == 0.5 and abs(x) <= 448.0 * s and (abs(x) > 224.0 * s)
    assert d.block_scale(np.zeros(3)) == 2.0 ** -126
    assert d.block_scale([np.inf, 1.0, -np.nan]) == d.block_scale([1.0])


def test_append_a_token_at_a_time_holds_what_one_call_holds():
    """With power-of-two scales a page filled in steps differs from one filled at once by subnormal codes only."""
    rng = np.random.default_rng(1)
    P, L = 16, 29
    x = rng.standard_normal((L, 2, 128)) * 2.0 ** rng.integers(-3, 4, (L, 1, 1))
    x = o.bf16_to_f64((np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16))
    table = np.array([[2, 0, -1]], np.int32)
    zero = np.zeros((3, 2, P, 128), np.uint8), np.full((3, 2), 9.0, np.float32)
    once = d.append(*zero, table, [L], [0, L], x)
    steps = zero
    for t in range(L):
        steps = d.append(*steps, table, [t + 1], [0, 1], x[t:t + 1])
    assert np.array_equal(once[1], steps[1])
    a, b = (o.e4m3_to_f64(c[0]) for c in (once, steps))
    assert np.all((a == b) | (np.abs(a) <= 2.0 ** -6))
    assert np.abs(a - b).max() <= 2.0 ** -8
    assert np.array_equal(once[0][1], zero[0][1]) and once[1][1, 0] == 9.0       # the page of nobody


def test_attention_by_loops():
    case = DenseCase(3, [21, 0, 5], [2, 1, 3], 16, 1, 2)
    mods = dict(softcap=3.0, slopes=case.slopes, prefix=np.array([20, 0, 1], np.int32))
    out, lse, *_ = case.oracle(0.1, **mods)
    for b in range(3):
        L = int(case.seq_lens[b])
        for i in range(int(case.q_lens[b])):
            r, pos = int(case.starts[b]) + i, L - int(case.q_lens[b]) + i
            for h in range(2):
                zs = []
                for s in range(L):
                    if s > pos and s >= mods["prefix"][b]:
                        continue
                    page, off = case.table[b, s // 16], s % 16
                    k = o.e4m3_to_f64(case.codes["k"][page, 0, off]) * float(case.scales["k"][page, 0])
                    z = 3.0 * math.tanh(0.1 * float(sum(k[j] * case.q[r, h, j] for j in range(128))) / 3.0)
                    zs.append((z - float(case.slopes[h]) * abs(pos - s),
                               o.e4m3_to_f64(case.codes["v"][page, 0, off]) * float(case.scales["v"][page, 0])))
                if not zs:
                    assert np.all(out[r, h] == 0) and lse[r, h] == -np.inf
                    continue
                total = sum(math.exp(z) for z, _ in zs)
                assert lse[r, h] == pytest.approx(math.log(total), rel=1e-12)
                np.testing.assert_allclose(out[r, h], sum(math.exp(z) * v for z, v in zs) / total, rtol=1e-10, atol=1e-13)


def test_step_plan_small():
    table = np.full((4, 3), -1, np.int32)
    table[0, 0] = 9
    lens, starts, slots, pos, count, after, refused = d.step_plan([3, 0, 0, 4], [2, 1, 40, 1], 4, table, [5, 6, 7, 8], 4, 6)
    assert refused == [2]                                   # 40 tokens need more pages than a table row has
    assert list(lens) == [5, 1, 0, 5] and list(starts) == [0, 2, 3, 3, 4]
    assert list(slots) == [9 * 4 + 3, 8 * 4, 7 * 4, 6 * 4, -1, -1] and list(pos) == [3, 4, 0, 4, -1, -1]
    assert count == 1 and after[0, 1] == 8 and after[1, 0] == 7 and after[3, 1] == 6
