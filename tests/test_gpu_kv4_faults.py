"""The rotating appends and the attention over the 4-bit cache on the GPU: inputs that were once answered wrongly."""
import numpy as np
import pytest

import workloads as wlm
from dense_cases import DenseCase, check_attention
from kv4_cases import Kv4Case, rope_table
from oracle import dense_oracle as d
from oracle import dsa_oracle as o
from oracle import kv4_oracle as f
from test_gpu_dense_edges import attend
from test_gpu_kv4_append import append, positions, same4, want4
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


@pytest.mark.parametrize("kind", [Kv4Case, DenseCase], ids=["4 bits", "8 bits"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_queries_of_requests_with_more_rows_than_tokens(kind, interleaved, in_place):
    """Attention answers all rows of such a request, so all its queries are written: rotated where the row has a position, and as
    they are in front of the first token.  Its keys are skipped."""
    import torch
    case = kind(48, [5, 0, 40, 33], [9, 7, 41, 2], 16, 1, 18, extra_rows=2)
    rope, pos = rope_table(45, 64), positions(case)
    live = np.arange(case.rows) < case.starts[-1]
    q = wlm.bits_to_torch(case.q_bits, "cuda")
    out = q if in_place else torch.full_like(q, -7.0)
    got, turned = append(case, rope, interleaved, q, out)
    want = np.where((pos >= 0)[:, None, None], f.rotate32(case.q, rope, np.maximum(pos, 0), interleaved), case.q)
    assert np.array_equal(turned[live], wlm.bf16_bits(want.astype(np.float32))[live])
    assert np.all(o.bf16_to_f64(turned[~live]) == (case.q[~live] if in_place else -7.0))
    if kind is Kv4Case:
        same4(case, got, want4(case, rope, interleaved))     # (the oracle skips such requests)
    else:
        k = f.rotate32(o.bf16_to_f64(case.new["k"]), rope, np.maximum(pos, 0), interleaved)
        codes, scales = d.append(case.codes["k"], case.scales["k"], case.table, case.seq_lens, case.starts, k.astype(np.float64))
        assert np.array_equal(got["ks"], scales) and np.array_equal(got["k"], codes)


def test_a_step_over_requests_with_more_rows_than_tokens():
    """Rows in front of the first token see a prefix, with queries that the append wrote into memory of its own."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(49, [5, 40, 33], [9, 41, 2], 16, 1, 6)
    rope, pos, prefix = rope_table(45, 128), positions(case), np.array([3, 20, 0], np.int32)
    cache, batch, q = case.gpu()
    k, v = (wlm.bits_to_torch(case.new[n], "cuda") for n in "kv")
    stale = torch.full_like(q, float("nan"))                # what a new tensor's memory may hold
    torch.cuda.synchronize()
    del stale
    turned = dsa.kv4_append(cache, batch, k, v, rope=dsa.RotaryTable.of(torch.from_numpy(rope).cuda()), q=q)
    case.q_bits = np.where((pos >= 0)[:, None, None], wlm.bf16_bits(f.rotate32(case.q, rope, np.maximum(pos, 0))), case.q_bits)
    assert np.array_equal(wlm.torch_to_bits(turned), case.q_bits)
    case.cache = want4(case, rope)
    got, lse = attend(case, (cache, batch, turned), prefix_lens=prefix)
    check_attention(got, lse, case.oracle(prefix=prefix))


@pytest.mark.parametrize("kind", [Kv4Case, DenseCase], ids=["4 bits", "8 bits"])
@pytest.mark.parametrize("starts,rows", [([0, 4, 9, 20], 12), ([-3, 2, 4, 6], 6), ([2, 4, 6, 8], 8), ([0, 4, 8, 12], 12)])
def test_requests_beside_those_whose_offsets_do_not_fit(kind, starts, rows):
    """Their keys, values and queries are written as ever; the others' rows are left alone."""
    import torch
    case = kind(50, [50, 33, 40], [4, 4, 4], 16, 2, 3)
    case.starts, case.rows = np.array(starts, np.int32), rows
    case.new = {n: wlm.bf16_bits(np.random.default_rng(50 + rows).standard_normal((rows, 2, 128)).astype(np.float32)) for n in "kv"}
    case.q_bits = wlm.bf16_bits(np.random.default_rng(51).standard_normal((rows, case.heads, 128)).astype(np.float32))
    pos = np.full(rows, -1)
    for b, L in enumerate(case.seq_lens):
        lo, hi = starts[b], starts[b + 1]
        if 0 <= lo and hi <= rows:
            pos[lo:hi] = L - (hi - lo) + np.arange(hi - lo)
    rope, good = rope_table(50, 96), pos >= 0
    assert 0 < good.sum()
    q = wlm.bits_to_torch(case.q_bits, "cuda")
    got, turned = append(case, rope, True, q, torch.full_like(q, -7.0))
    k = f.rotate32(o.bf16_to_f64(case.new["k"]), rope, np.maximum(pos, 0), True)
    assert np.array_equal(turned[good], wlm.bf16_bits(f.rotate32(case.q, rope, np.maximum(pos, 0), True))[good])
    assert np.all(o.bf16_to_f64(turned[~good]) == -7.0)
    if kind is Kv4Case:
        same4(case, got, f.append(case.cache, case.table, case.seq_lens, case.starts, k, o.bf16_to_f64(case.new["v"])))
    else:
        for name, x in (("k", k.astype(np.float64)), ("v", o.bf16_to_f64(case.new["v"]))):
            codes, scales = np.array(case.codes[name]), np.array(case.scales[name])
            for b in range(3):                               # a request whose offsets fit, by itself
                lo, hi = starts[b], starts[b + 1]
                if 0 <= lo and hi <= rows:
                    codes, scales = d.append(codes, scales, case.table[b:b + 1], case.seq_lens[b:b + 1], np.array([0, hi - lo]), x[lo:hi])
            assert np.array_equal(got[name + "s"], scales) and np.array_equal(got[name], codes), name
