"""The 4-bit K/V append and the rotation of both appends on the GPU against the oracle: codes and scales, equal."""
import numpy as np
import pytest

import workloads as wlm
from dense_cases import DenseCase
from kv4_cases import Kv4Case, rope_table
from oracle import dense_oracle as d
from oracle import dsa_oracle as o
from oracle import kv4_oracle as f
from test_gpu_kv8_append import before

pytestmark = pytest.mark.gpu


def put(a):
    import torch
    return torch.from_numpy(np.array(a)).cuda()


def positions(case):
    """Position of each row; -1 behind the last request's."""
    pos = np.full(case.rows, -1)
    for b, (L, n) in enumerate(zip(case.seq_lens, case.q_lens)):
        pos[case.starts[b]:case.starts[b + 1]] = L - n + np.arange(n)
    return pos


def append(case, rope=None, interleaved=False, q=None, q_out=None, k=None, v=None, batch=None):
    """Appends on the device; (the cache, rotated q or None) as numpy."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    cache, default, _ = case.gpu()
    four = isinstance(case, Kv4Case)
    k = wlm.bits_to_torch(case.new["k"], "cuda") if k is None else k
    v = wlm.bits_to_torch(case.new["v"], "cuda") if v is None else v
    table = None if rope is None else dsa.RotaryTable.of(put(rope), interleaved)
    turned = (dsa.kv4_append if four else dsa.kv8_append)(cache, batch or default, k, v, rope=table, q=q, q_out=q_out)
    torch.cuda.synchronize()
    got = {"k": cache.k_codes.cpu().numpy(), "v": cache.v_codes.cpu().numpy(), "ks": cache.k_scales.cpu().numpy(),
           "vs": cache.v_scales.float().cpu().numpy().astype(np.float64)}
    return got, None if turned is None else wlm.torch_to_bits(turned)


def want4(case, rope=None, interleaved=False):
    k = o.bf16_to_f64(case.new["k"])
    if rope is not None:
        k = f.rotate32(k, rope, np.maximum(positions(case), 0), interleaved)
    return f.append(case.cache, case.table, case.seq_lens, case.starts, k, o.bf16_to_f64(case.new["v"]))


def same4(case, got, want):
    assert np.array_equal(got["ks"], want["ks"]), "K scales"
    assert np.array_equal(got["vs"], want["vs"], equal_nan=True), "V scales"
    ok = np.repeat(want["ks"] != f.NAN_SCALE, 16, -1)        # codes under a NaN scale are unspecified
    assert np.array_equal(got["k"][ok], want["k"][ok]), "K codes"
    ok = ~np.isnan(want["vs"])
    assert np.array_equal(got["v"][ok], want["v"][ok]), "V codes"


CASES = [
    ([1], [1], 16, 1), ([64], [64], 64, 2), ([65, 1, 300], [1, 1, 1], 64, 2), ([640, 5, 1000, 33], [4, 5, 130, 1], 128, 2),
    ([100, 0, 41, 17], [37, 0, 17, 1], 16, 3), ([31, 32, 33, 200], [2, 1, 33, 0], 32, 4), ([40], [3], 16, 9),
]


@pytest.mark.parametrize("n", range(len(CASES)))
def test_matches_the_oracle(n):
    seq, new, P, kv = CASES[n]
    case = Kv4Case(300 + n, seq, new, P, kv, 1, extra_rows=n % 3)
    got, _ = append(case)
    same4(case, got, want4(case))


@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [2, 4])
def test_rotated_keys_and_queries(n, dim, interleaved):
    import torch
    seq, new, P, kv = CASES[n]
    case = Kv4Case(320 + n, seq, new, P, kv, 5, extra_rows=2)
    rope, pos = rope_table(max(seq) + 3, dim), positions(case)
    q = wlm.bits_to_torch(case.q_bits, "cuda")
    out = torch.full_like(q, -7.0)
    got, turned = append(case, rope, interleaved, q, out)
    same4(case, got, want4(case, rope, interleaved))
    live = pos >= 0
    want = f.rotate32(case.q, rope, np.maximum(pos, 0), interleaved)
    assert np.array_equal(turned[live], wlm.bf16_bits(want)[live])
    assert np.all(o.bf16_to_f64(turned[~live]) == -7.0)


@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [0, 2, 3, 4, 5])
def test_the_8_bit_append_with_rotation(n, dim, interleaved):
    import torch
    seq, new, P, kv = CASES[n]
    case = before(DenseCase(340 + n, seq, new, P, kv, 3, extra_rows=n % 3))
    rope, pos = rope_table(max(seq), dim), positions(case)
    q = wlm.bits_to_torch(case.q_bits, "cuda")
    out = torch.full_like(q, -7.0)
    got, turned = append(case, rope, interleaved, q, out)
    k = f.rotate32(o.bf16_to_f64(case.new["k"]), rope, np.maximum(pos, 0), interleaved)
    for name, x in (("k", k.astype(np.float64)), ("v", o.bf16_to_f64(case.new["v"]))):
        codes, scales = d.append(case.codes[name], case.scales[name], case.table, case.seq_lens, case.starts, x)
        assert np.array_equal(got[name + "s"], scales), name + " scales"
        assert np.array_equal(got[name], codes), name + " codes"
    live = pos >= 0
    assert np.array_equal(turned[live], wlm.bf16_bits(f.rotate32(case.q, rope, np.maximum(pos, 0), interleaved))[live])
    assert np.all(o.bf16_to_f64(turned[~live]) == -7.0)


def test_scales_at_their_limits_zeros_infinities_and_nan():
    case = Kv4Case(350, [40], [9], 16, 1, 1)
    k, v = case.new["k"], case.new["v"]
    for x in (k, v):
        x[0] = 0
        x[1] = 0x8000                                        # -0
        x[2] = 0x0001                                        # the smallest
        x[3] = 0x7F7F                                        # the largest
        x[4, 0, ::2] = 0x7F80                                # infinities beside finite values
        x[5, 0, 40] = 0xFF80
        x[6, 0, 3] = 0x7FC0                                  # NaN
        x[7, 0, 64:] = 0x7F80                                # blocks of infinities alone
        x[8] = wlm.bf16_bits(np.linspace(-6, 6, 128).astype(np.float32))   # ties among them
    got, _ = append(case)
    same4(case, got, want4(case))
    page, off = case.table[0, 37 // 16], 37 % 16             # row 6
    assert got["ks"][page, 0, off].tolist()[0] == 255 and 255 not in got["ks"][page, 0, off][1:] and np.isnan(got["vs"][page, 0, off])


def test_rows_of_a_fused_projection_and_queries_rotated_in_place():
    import torch
    case = Kv4Case(360, [50, 33], [18, 1], 16, 2, 3)
    wide = torch.full((case.rows, case.heads + 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    h = case.heads
    wide[:, :h] = wlm.bits_to_torch(case.q_bits, "cuda")
    wide[:, h:h + 2] = wlm.bits_to_torch(case.new["k"], "cuda")
    wide[:, h + 2:] = wlm.bits_to_torch(case.new["v"], "cuda")
    rope = rope_table(60, 64)
    got, _ = append(case, rope, False, wide[:, :h], wide[:, :h], wide[:, h:h + 2], wide[:, h + 2:])
    same4(case, got, want4(case, rope))
    assert np.array_equal(wlm.torch_to_bits(wide[:, :h].contiguous()), wlm.bf16_bits(f.rotate32(case.q, rope, positions(case))))
    assert np.array_equal(wlm.torch_to_bits(wide[:, h:h + 2].contiguous()), case.new["k"])     # k itself stays


def test_decode_rows_without_offsets():
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(370, [50, 0, 33], [1, 0, 1], 16, 2, 3)
    case.starts = np.arange(4, dtype=np.int32)
    case.rows, case.q_lens = 3, np.array([1, 1, 1])
    rng = np.random.default_rng(1)
    case.new = {n: wlm.bf16_bits(rng.standard_normal((3, 2, 128)).astype(np.float32)) for n in "kv"}
    batch = dsa.Batch(put(case.table), put(case.seq_lens), None, max_seq_len=50)
    rope = rope_table(50, 128)
    got, _ = append(case, rope, batch=batch)
    case.q_lens = np.array([1, 0, 1])                        # the empty request's row has no position
    want = dict(case.cache)
    for r, (b, pos) in enumerate(((0, 49), (None, None), (2, 32))):
        if b is None:
            continue
        at = case.table[b, pos // 16], slice(None), pos % 16
        k = f.rotate32(o.bf16_to_f64(case.new["k"])[r:r + 1], rope, np.array([pos]))[0]
        for h in range(2):
            want["k"][at[0], h, at[2]], want["ks"][at[0], h, at[2]] = f.quantise_k(k[h])
            want["v"][at[0], h, at[2]], want["vs"][at[0], h, at[2]] = f.quantise_v(o.bf16_to_f64(case.new["v"])[r, h])
    same4(case, got, want)


@pytest.mark.parametrize("rotated", [False, True])
def test_out_of_range_pages_and_rows_behind_the_last_are_skipped(rotated):
    case = Kv4Case(380, [50, 33], [20, 2], 16, 2, 1, extra_rows=5)
    case.table[0, 2], case.table[1, 2] = case.pages, -1
    rope = rope_table(50, 64) if rotated else None
    got, _ = append(case, rope)
    same4(case, got, want4(case, rope))


@pytest.mark.parametrize("starts,rows", [([0, 5, 3, 8], 8), ([0, 4, 9, 20], 12), ([-3, 2, 4, 6], 6), ([2, 4, 6, 8], 8)])
def test_offsets_that_do_not_fit_the_batch_are_skipped(starts, rows):
    case = Kv4Case(390, [50, 33, 40], [4, 4, 4], 16, 2, 1)
    case.starts, case.rows = np.array(starts, np.int32), rows
    case.new = {n: wlm.bf16_bits(case.rng.standard_normal((rows, 2, 128)).astype(np.float32)) for n in "kv"}
    got, _ = append(case)
    touched = np.zeros(got["vs"].shape, bool)                # only slots of requests whose offsets make sense may change
    for b, L in enumerate(case.seq_lens):
        lo, hi = starts[b], starts[b + 1]
        if 0 <= lo < hi <= rows:
            for pos in range(int(L) - (hi - lo), int(L)):
                touched[case.table[b, pos // 16], :, pos % 16] = True
    for n in ("k", "v", "ks"):
        assert np.array_equal(got[n][~touched], case.cache[n][~touched]), n
    assert np.array_equal(got["vs"][~touched], case.cache["vs"][~touched], equal_nan=True)
