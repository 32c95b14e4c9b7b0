"""The block-scaled 8-bit K/V append on the GPU against the oracle: codes and scales, equal."""
import numpy as np
import pytest

import workloads as wlm
from dense_cases import DenseCase
from oracle import dense_oracle as d
from oracle import dsa_oracle as o

pytestmark = pytest.mark.gpu


def before(case):
    """The case's pool as it was before this step's tokens: their slots hold what a recycled page may hold."""
    for b, L in enumerate(case.seq_lens):
        for s in range(int(L - case.q_lens[b]), int(L)):
            for n in "kv":
                case.codes[n][case.table[b, s // case.P], :, s % case.P] = 0x33
    return case


def run(case, k=None, v=None):
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    cache, batch, _ = case.gpu()
    k = wlm.bits_to_torch(case.new["k"], "cuda") if k is None else k
    v = wlm.bits_to_torch(case.new["v"], "cuda") if v is None else v
    dsa.kv8_append(cache, batch, k, v)
    torch.cuda.synchronize()
    return {"k": (cache.k_codes.cpu().numpy(), cache.k_scales.cpu().numpy()), "v": (cache.v_codes.cpu().numpy(), cache.v_scales.cpu().numpy())}


def check(case, got):
    for n in "kv":
        codes, scales = d.append(case.codes[n], case.scales[n], case.table, case.seq_lens, case.starts, o.bf16_to_f64(case.new[n]))
        assert np.array_equal(got[n][1], scales), n + " scales"
        assert np.array_equal(got[n][0], codes), n + " codes"


CASES = [
    ([1], [1], 16, 1), ([64], [64], 64, 2), ([65, 1, 300], [1, 1, 1], 64, 2), ([640, 5, 1000, 33], [4, 5, 130, 1], 128, 2),
    ([100, 0, 41, 17], [37, 0, 17, 1], 16, 3), ([31, 32, 33, 200], [2, 1, 33, 0], 32, 4),
]


@pytest.mark.parametrize("n", range(len(CASES)))
def test_matches_the_oracle(n):
    seq, new, P, kv = CASES[n]
    case = before(DenseCase(300 + n, seq, new, P, kv, 1, extra_rows=n % 3))
    check(case, run(case))


@pytest.mark.parametrize("P", [16, 64])
def test_pages_are_recoded_when_a_scale_grows_and_keep_theirs_when_it_does_not(P):
    case = before(DenseCase(7, [P - 3, P - 3, 2 * P - 5], [2, 2, 3], P, 2, 1))
    x = o.bf16_to_f64(case.new["k"])
    x[:2] *= 64.0
    x[2:] /= 64.0
    case.new["k"] = wlm.bf16_bits(x.astype(np.float32))
    got = run(case)
    check(case, got)
    page = case.table[0, 0]
    assert np.all(got["k"][1][page] > case.scales["k"][page]) and np.any(got["k"][0][page, :, 0] != case.codes["k"][page, :, 0])
    page = case.table[1, 0]
    assert np.array_equal(got["k"][1][page], case.scales["k"][page])


def test_scales_that_are_no_powers_of_two_are_kept_or_left():
    case = before(DenseCase(8, [20, 21], [1, 2], 32, 2, 1))
    case.scales["k"] *= np.float32(1.37)
    case.scales["v"] *= np.float32(0.011)
    check(case, run(case))


def test_zeros_infinities_and_nan():
    case = before(DenseCase(9, [16, 5, 40], [16, 1, 2], 16, 1, 1))
    bits = case.new["k"]
    bits[:] = 0
    bits[16, 0, 3] = 0x7F80
    bits[16, 0, 4] = 0xFF80
    bits[17, 0, 0] = 0x7FC0
    bits[17, 0, 1] = 0x3F80
    bits[18, 0, :] = 0x0001
    got = run(case)
    check(case, got)
    assert got["k"][1][case.table[0, 0], 0] == 2.0 ** -126
    assert got["k"][0][case.table[2, 2], 0, 6, 0] == 0x7F


def test_rows_of_a_fused_projection():
    import torch
    case = before(DenseCase(10, [50, 33], [18, 1], 16, 2, 1))
    wide = torch.full((case.rows, 6, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:3] = wlm.bits_to_torch(case.new["k"], "cuda")
    wide[:, 4:6] = wlm.bits_to_torch(case.new["v"], "cuda")
    check(case, run(case, wide[:, 1:3], wide[:, 4:6]))


def test_out_of_range_pages_and_rows_behind_the_last_are_skipped():
    case = before(DenseCase(11, [50, 33], [20, 2], 16, 2, 1, extra_rows=5))
    case.table[0, 2], case.table[1, 2] = case.pages, -1
    check(case, run(case))


def test_refusals():
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = DenseCase(12, [50], [3], 16, 2, 1)
    cache, batch, _ = case.gpu()
    k = wlm.bits_to_torch(case.new["k"], "cuda")
    for bad in (k.float(), k[:, :1], k[:2], k.transpose(1, 2).contiguous().transpose(1, 2), k.cpu()):
        with pytest.raises(ValueError):
            dsa.kv8_append(cache, batch, bad, k)
    odd = torch.zeros(3 * 257, dtype=torch.bfloat16, device="cuda").as_strided((3, 2, 128), (257, 128, 1))
    with pytest.raises(dsa.DsaError, match="stride"):
        dsa.kv8_append(cache, batch, odd, k)
