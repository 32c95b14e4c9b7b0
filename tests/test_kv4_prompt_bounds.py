"""The bound of many rows over the 4-bit cache is tighter than 8-bit probabilities or rounded values, planted in the oracle's place."""
import numpy as np
import pytest

from kv4_cases import Kv4Case
from kv4_prompt_bounds import prompt_errors
from oracle import dsa_oracle as o
from oracle import kv4_oracle as f

import workloads as wlm

SCALE = 2.0 ** -9


def significand(x, bits):
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


def rows(case, p_bits, v_bits):
    """Outputs of one request's whole prompt with p and V of so many bits, in bf16."""
    L, s = int(case.seq_lens[0]), np.arange(int(case.seq_lens[0]))
    pages = case.table[0, s // case.P]
    k = f.values(case.cache["k"][pages, 0, s % case.P]) * np.repeat(np.exp2(case.cache["ks"][pages, 0, s % case.P].astype(np.float64) - 127), 32, -1)
    v = f.values(case.cache["v"][pages, 0, s % case.P]) * case.cache["vs"][pages, 0, s % case.P][:, None]
    out = np.zeros((L, case.heads, 128))
    for h in range(case.heads):
        z = SCALE * case.q[:, h] @ k.T
        z[s[None] > s[:, None]] = -np.inf
        p = np.exp(z - z.max(1, keepdims=True))
        out[:, h] = significand(p, p_bits) @ significand(v, v_bits) / p.sum(1, keepdims=True)
    return o.bf16_to_f64(wlm.bf16_bits(out.astype(np.float32)))


@pytest.mark.parametrize("p_bits,v_bits,good", [(11, 11, True), (53, 53, True), (8, 11, False), (11, 8, False)])
def test_what_the_bound_tells_apart(p_bits, v_bits, good):
    case = Kv4Case(60, [70], [70], 16, 1, 8)
    over = prompt_errors(case, rows(case, p_bits, v_bits), case.oracle(scale=SCALE), SCALE).max()
    assert (over <= 1.0) == good, over
