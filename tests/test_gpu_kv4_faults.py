"""The rotating appends and the attention over the 4-bit cache on the GPU: inputs that were once answered wrongly."""
import numpy as np
import pytest

import workloads as wlm
from dense_cases import check_attention
from kv4_cases import Kv4Case
from oracle import kv4_oracle as f
from test_gpu_dense_edges import attend
from test_gpu_kv4_append import want4
from test_gpu_kv4_edges import BOTH

pytestmark = pytest.mark.gpu


@BOTH
def test_scales_of_v_above_those_of_the_8_bit_cache(shape):
    """As test_values_of_any_size, for scales up to 2^125, and with biases that take most probabilities to 0."""
    case = Kv4Case(45, *shape, spread=0.0)
    slopes = np.full(case.heads, 2.0, np.float32)            # keys 100 away score -200 and less: p is 0
    want, biased = case.oracle(), case.oracle(slopes=slopes)
    assert np.nanmax(case.cache["vs"]) < 2.0                 # outputs below 6 * 2^125: bf16 holds them
    case.cache["vs"] = np.ldexp(case.cache["vs"], 124)
    got, lse = attend(case)
    check_attention(np.ldexp(got, -124), lse, want)
    got, lse = attend(case, slopes=slopes)
    check_attention(np.ldexp(got, -124), lse, biased, reach=2.0 * 300)


@BOTH
def test_the_largest_values_that_an_append_takes(shape):
    """V's rows up to bf16's largest number, appended and attended to."""
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(46, *shape)
    rng = np.random.default_rng(46)
    v = rng.standard_normal((case.rows, case.kv, 128)) * 2.0 ** rng.integers(100, 127, (case.rows, case.kv, 1))
    bits = wlm.bf16_bits(np.clip(v, -3e38, 3e38).astype(np.float32))
    bits[::3, 0, 5:9] = 0x7F7F                               # the largest, and its negative
    bits[1::3, 1, 40] = 0xFF7F
    case.new["v"] = bits
    cache, batch, q = case.gpu()
    dsa.kv4_append(cache, batch, wlm.bits_to_torch(case.new["k"], "cuda"), wlm.bits_to_torch(bits, "cuda"))
    case.cache = want4(case)
    assert np.nanmax(case.cache["vs"]) > 2.0 ** 125
    got, lse = attend(case, (cache, batch, q))
    check_attention(got, lse, case.oracle())


def test_one_token_of_the_largest_value():
    case = Kv4Case(47, [1, 1], [1, 1], 16, 1, 8)
    for b in range(2):
        at = case.table[b, 0], 0, 0
        case.cache["v"][at], case.cache["vs"][at] = f.quantise_v(np.full(128, 255 * 2.0 ** 120))
    got, lse = attend(case)
    assert np.all(got == 255 * 2.0 ** 120)                   # bf16's largest number
