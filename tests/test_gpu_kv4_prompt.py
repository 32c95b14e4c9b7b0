"""Attention of many rows over the 4-bit cache on the GPU to the precision that it documents: 11 bits of p, V exact."""
import numpy as np
import pytest

from kv4_cases import Kv4Case
from kv4_prompt_bounds import prompt_errors
from test_gpu_dense_edges import attend

pytestmark = pytest.mark.gpu

SCALE = 2.0 ** -9                                            # small scores: their errors are well below p's


@pytest.mark.parametrize("seq,new,P,kv,group", [([70], [70], 16, 1, 8), ([129, 40, 257], [129, 40, 257], 64, 2, 4), ([300, 90], [20, 66], 32, 1, 16),
                                                ([5, 70], [5, 3], 16, 1, 64), ([1500], [70], 128, 1, 8)])
def test_probabilities_keep_11_bits(seq, new, P, kv, group):
    case = Kv4Case(60, seq, new, P, kv, group)
    assert min(new) * group > 64
    got, _ = attend(case, scale=SCALE)
    over = prompt_errors(case, got, case.oracle(scale=SCALE), SCALE)
    assert over.max() <= 1.0, f"off by {over.max():.3f} of the bound"


@pytest.mark.parametrize("down,v_error", [(26, 0.0), (30, 2.0 ** -34)])
def test_values_of_rows_that_do_not_see_the_largest_scale(down, v_error):
    """Key 20 holds V's largest scale, and the rows before it see only scales of 2^-down of it."""
    case = Kv4Case(61, [40, 60], [40, 60], 32, 2, 8)
    rng = np.random.default_rng(61)
    for b, L in enumerate(case.seq_lens):
        s = np.arange(int(L))
        case.cache["vs"][case.table[b, s // 32], :, s % 32] = (1 + rng.integers(0, 128, (len(s), 2)) / 128) * 2.0 ** -down
        case.cache["vs"][case.table[b, 0], :, 20] = 1.0
    got, _ = attend(case, scale=SCALE)
    over = prompt_errors(case, got, case.oracle(scale=SCALE), SCALE, v_error)
    assert over.max() <= 1.0, f"off by {over.max():.3f} of the bound"
