"""The oracle of the rotation, the 4-bit cache and the attention over it, against brute force and closed forms (CPU)."""
import math

import numpy as np
import pytest

import workloads as wlm
from kv4_cases import Kv4Case, rope_table
from oracle import dsa_oracle as o
from oracle import kv4_oracle as f


def test_the_16_values():
    """e2m1 by its fields: sign, two bits of exponent (bias 1) and one of mantissa."""
    for c in range(16):
        s, e, m = -1.0 if c & 8 else 1.0, c >> 1 & 3, c & 1
        assert f.E2M1[c] == s * (m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))
    packed = np.arange(256, dtype=np.uint8)[None]
    assert np.array_equal(f.values(packed)[0, 0::2], f.E2M1[np.arange(256) & 15])
    assert np.array_equal(f.values(packed)[0, 1::2], f.E2M1[np.arange(256) >> 4])
    codes = np.arange(16, dtype=np.uint8)
    assert np.array_equal(f.values(f.two_a_byte(codes)), f.E2M1)
    assert np.array_equal(f.encode(f.E2M1), codes)


def test_codes_are_the_nearest_ties_to_even_saturating():
    x = np.concatenate([np.linspace(-7, 7, 4001), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 100.0, -np.inf]])
    got = f.E2M1[f.encode(x)]
    err = np.abs(got - np.clip(x, -6, 6))
    for v in f.E2M1:
        assert np.all(err <= np.abs(v - np.clip(x, -6, 6)))
    assert f.E2M1[f.encode([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    assert f.E2M1[f.encode([100.0, -np.inf])].tolist() == [6.0, -6.0]


def test_block_exponents_are_the_smallest_that_hold_the_block():
    rng = np.random.default_rng(0)
    for x in list(rng.standard_normal(60) * 2.0 ** rng.uniform(-8, 12, 60)) + [6.0, 6.0001, 5.9999, 3.0, 3.0001, 1.5 * 2.0 ** 9]:
        e = f.block_exponent([x, x / 3])
        assert abs(x) <= 6.0 * 2.0 ** e and abs(x) > 3.0 * 2.0 ** e
        assert e == math.ceil(math.log2(abs(x) / 6.0))
    assert f.block_exponent(np.zeros(3)) == -15 and f.block_exponent([1e-9]) == -15 and f.block_exponent([1e9]) == 13
    assert f.block_exponent([np.inf, 1.0, -np.nan]) == f.block_exponent([1.0])


def test_v_scales_are_bf16_to_nearest_even_with_a_floor():
    rng = np.random.default_rng(1)
    for x in np.abs(rng.standard_normal(200)) * 2.0 ** rng.uniform(-100, 100, 200):
        assert f._bf16(float(np.float32(x))) == float(o.bf16_to_f64(wlm.bf16_bits(np.array([x], np.float32)))[0])
    assert f.quantise_v(np.zeros(128))[1] == 2.0 ** -126
    x = np.zeros(128)
    x[3], x[5] = np.nan, 12.0
    codes, s = f.quantise_v(x)
    assert math.isnan(s) and f.values(codes)[5] == 6.0 and f.values(codes)[3] == 0.0
    codes, scales = f.quantise_k(np.where(np.arange(128) == 40, np.nan, 1.0))
    assert scales.tolist() == [125, f.NAN_SCALE, 125, 125] and f.values(codes)[40] == 0.0 and f.values(codes)[41] == 4.0


def test_what_the_quantisers_keep():
    """Half of the largest step, 2 * scale / 2, and what bf16 takes from a scale that is rounded down."""
    rng = np.random.default_rng(2)
    for _ in range(50):
        x = rng.standard_normal(128) * 2.0 ** rng.uniform(-6, 6)
        codes, scales = f.quantise_k(x)
        s = np.repeat(2.0 ** (scales.astype(float) - 127), 32)
        assert np.all(np.abs(f.values(codes) * s - x) <= s)
        codes, s = f.quantise_v(x)
        assert np.all(np.abs(f.values(codes) * s - x) <= s * (1 + 6 * 2.0 ** -8))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [32, 96, 128])
def test_the_rotation_is_that_of_complex_numbers(dim, interleaved):
    rng = np.random.default_rng(dim)
    x, table, pos = rng.standard_normal((9, 3, 128)), rope_table(50, dim), rng.integers(0, 50, 9)
    got = f.rotate(x, table, pos, interleaved)
    for i in range(dim // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + dim // 2)
        z = (x[..., a] + 1j * x[..., b]) * (table[pos, i].astype(float) + 1j * table[pos, dim // 2 + i])[:, None]
        assert np.allclose(got[..., a], z.real, rtol=0, atol=1e-12) and np.allclose(got[..., b], z.imag, rtol=0, atol=1e-12)
    assert np.array_equal(got[..., dim:], x[..., dim:])
    # three roundings to 24 bits of values no larger than the pair
    assert np.abs(f.rotate32(x.astype(np.float32), table, pos, interleaved) - f.rotate(x.astype(np.float32), table, pos, interleaved)).max() <= \
        3 * 2.0 ** -24 * 2 * np.abs(x).max()


def test_scores_of_rotated_pairs_depend_on_their_distance():
    rng = np.random.default_rng(3)
    q, k, table = rng.standard_normal((1, 1, 128)), rng.standard_normal((1, 1, 128)), rope_table(100, 128)
    dots = [float((f.rotate(q, table, np.array([n + 7])) * f.rotate(k, table, np.array([n]))).sum()) for n in (0, 5, 60, 92)]
    assert np.ptp(dots) <= 1e-5                              # the table's float32
    assert abs(dots[0] - float((q * k).sum())) > 1e-2


def test_append_a_token_at_a_time_is_one_append():
    rng = np.random.default_rng(4)
    P, L = 16, 29
    k, v = rng.standard_normal((2, L, 2, 128)) * 2.0 ** rng.integers(-3, 4, (2, L, 1, 1))
    table = np.array([[2, 0, -1]], np.int32)
    zero = {"k": np.zeros((3, 2, P, 64), np.uint8), "v": np.zeros((3, 2, P, 64), np.uint8), "ks": np.zeros((3, 2, P, 4), np.uint8), "vs": np.zeros((3, 2, P))}
    once, steps = f.append(zero, table, [L], [0, L], k, v), zero
    for t in range(L):
        steps = f.append(steps, table, [t + 1], [0, 1], k[t:t + 1], v[t:t + 1])
    assert all(np.array_equal(once[n], steps[n]) for n in zero)
    assert not once["k"][1].any() and not once["vs"][0, :, L - P:].any()
    assert np.array_equal(once["k"][0, 1, 3], f.quantise_k(k[19, 1])[0]) and once["vs"][0, 1, 3] == f.quantise_v(v[19, 1])[1]


def test_attention_by_loops():
    case = Kv4Case(3, [21, 0, 5], [2, 1, 3], 16, 1, 2)
    mods = dict(softcap=3.0, slopes=case.slopes, prefix=np.array([20, 0, 1], np.int32))
    out, lse, *_ = case.oracle(0.1, **mods)
    c = case.cache
    for b in range(3):
        L = int(case.seq_lens[b])
        for i in range(int(case.q_lens[b])):
            r, pos = int(case.starts[b]) + i, L - int(case.q_lens[b]) + i
            for h in range(2):
                zs = []
                for s in range(L):
                    if s > pos and s >= mods["prefix"][b]:
                        continue
                    at = case.table[b, s // 16], 0, s % 16
                    dot = 0.0
                    for j in range(128):
                        code = int(c["k"][at][j // 2]) >> (4 * (j % 2)) & 15
                        dot += float(f.E2M1[code]) * 2.0 ** (int(c["ks"][at][j // 32]) - 127) * float(case.q[r, h, j])
                    z = 3.0 * math.tanh(0.1 * dot / 3.0)
                    zs.append((z - float(case.slopes[h]) * abs(pos - s), f.values(c["v"][at]) * float(c["vs"][at])))
                if not zs:
                    assert np.all(out[r, h] == 0) and lse[r, h] == -np.inf
                    continue
                total = sum(math.exp(z) for z, _ in zs)
                assert abs(lse[r, h] - math.log(total)) <= 1e-10
                assert np.allclose(out[r, h], sum(math.exp(z) / total * x for z, x in zs), rtol=0, atol=1e-10)
