"""Dense attention over the 4-bit cache on the GPU where it can go wrong: masked and visible NaN, wide scales, bad pages, rows
that are left alone, long and many requests, strides, streams, graphs and stale workspaces.  Every case runs in the kernel for
few rows and, with more than 64 rows * heads a request, in the one for prompts."""
import numpy as np
import pytest

import workloads as wlm
from dense_cases import check_attention
from kv4_cases import Kv4Case, rope_table
from oracle import dsa_oracle as o
from oracle import kv4_oracle as f
from test_gpu_dense_edges import attend, put, row_limits

pytestmark = pytest.mark.gpu

DECODE = ([300, 77, 129], [1, 3, 2], 32, 2, 8)
PROMPT = ([300, 77, 129], [45, 9, 129], 32, 2, 8)
BOTH = pytest.mark.parametrize("shape", [DECODE, PROMPT], ids=["decode", "prompt"])


def at(case, b, key, h):
    return case.table[b, key // case.P], h, key % case.P


@BOTH
@pytest.mark.parametrize("what", ["nan", "infinity"])
def test_a_v_scale_that_is_not_finite_reaches_the_rows_that_see_it(shape, what):
    case = Kv4Case(1, *shape)
    want = [np.array(x) for x in case.oracle()]
    limit, req = row_limits(case)
    bad = np.zeros((case.rows, case.heads), bool)
    for b, key, h in ((0, 12, 1), (0, 298, 0), (1, 76, 0), (2, 127, 1), (2, 128, 1)):
        case.cache["vs"][at(case, b, key, h)] = np.nan if what == "nan" else np.inf
        bad[np.ix_((req == b) & (limit > key), range(h * case.group, (h + 1) * case.group))] = True
    got, lse = attend(case)
    # (an infinite scale is not one that the cache may hold: its rows are not finite, and no others change)
    assert np.all(~np.isfinite(got[bad]).any(-1)) if what == "infinity" else np.all(np.isnan(got[bad]))
    assert np.all(np.isfinite(got[~bad]))
    check_attention(np.where(bad[..., None], want[0], got), lse, want)


@BOTH
def test_a_nan_scale_in_k_reaches_the_rows_that_see_it(shape):
    case = Kv4Case(2, *shape)
    want = [np.array(x) for x in case.oracle()]
    limit, req = row_limits(case)
    bad = np.zeros((case.rows, case.heads), bool)
    for b, key, h in ((0, 299, 1), (1, 74, 0), (2, 100, 1)):
        case.cache["ks"][at(case, b, key, h)][key % 4] = f.NAN_SCALE
        bad[np.ix_((req == b) & (limit > key), range(h * case.group, (h + 1) * case.group))] = True
    got, lse = attend(case)
    assert np.array_equal(np.isnan(lse), bad) and np.array_equal(np.isnan(got), np.broadcast_to(bad[..., None], got.shape))
    want[4] = np.where(bad, np.nan, want[4])                 # what the check leaves out
    check_attention(got, np.where(bad, 0.0, lse), want)


@BOTH
def test_a_query_that_is_not_finite_poisons_its_own_pair_only(shape):
    case = Kv4Case(3, *shape)
    want = [np.array(x) for x in case.oracle()]
    bad = np.zeros((case.rows, case.heads), bool)
    for r, h, bits in ((0, 3, 0x7FC0), (2, 15, 0x7F80), (case.rows - 1, 0, 0xFF80)):
        case.q_bits[r, h, 9] = bits
        bad[r, h] = True
    got, lse = attend(case)
    assert np.array_equal(np.isnan(lse), bad) and np.array_equal(np.isnan(got), np.broadcast_to(bad[..., None], got.shape))
    want[4] = np.where(bad, np.nan, want[4])
    check_attention(got, np.where(bad, 0.0, lse), want)


@BOTH
def test_scales_far_apart_at_their_limits_and_of_zero(shape):
    case = Kv4Case(4, *shape)
    rng = np.random.default_rng(4)
    case.cache["vs"] *= np.exp2(rng.integers(-12, 13, case.cache["vs"].shape))
    ks = case.cache["ks"]
    ks[ks != f.NAN_SCALE] = rng.integers(127 - 15, 127 + 1, (ks != f.NAN_SCALE).sum())
    ks[case.table[0, 2]] = 127 - 15
    case.cache["vs"][case.table[0, 1]] = 0.0
    case.cache["vs"][case.table[1, :3], 1] = 0.0             # a request and head whose values are all zero
    got, lse = attend(case)
    check_attention(got, lse, case.oracle())
    assert np.all(got[case.starts[1]:case.starts[2], case.group:] == 0.0)
    ks[ks != f.NAN_SCALE] = 127 + 13                         # the largest: scores of 2^13 and more, one key each
    q = case.q * 2.0 ** -16
    case.q_bits = wlm.bf16_bits(q.astype(np.float32))
    got, lse = attend(case)
    check_attention(got, lse, case.oracle())


@BOTH
@pytest.mark.parametrize("k", [-119, -60, 60, 119])
def test_values_of_any_size(shape, k):
    """V's scales from 2^-126 to 2^120: the output is that of scales near one, times a power of two, up to the rounding of
    bf16's subnormal numbers."""
    case = Kv4Case(5, *shape, spread=0.0)
    out, lse, A, C, Z = case.oracle()
    assert 2.0 ** -7 <= np.nanmin(case.cache["vs"]) and np.nanmax(case.cache["vs"]) < 2.0
    case.cache["vs"] = np.ldexp(case.cache["vs"], k)
    got, got_lse = attend(case)
    C = C + 2.0 ** 18 * 2.0 ** (-134 - k)                    # half a step of those numbers (the bound takes 2^-18 of C)
    check_attention(np.ldexp(got, -k), got_lse, (out, lse, A, C, Z))


def test_a_token_that_only_later_rows_see_leaves_the_others_alone():
    case = Kv4Case(21, [65, 131], [3, 4], 16, 2, 8)
    case.cache["vs"] *= 2.0 ** -30
    for b, L in enumerate(case.seq_lens):
        case.cache["vs"][case.table[b, (L - 1) // 16], :, (L - 1) % 16] = 2.0 ** 118
    out, lse, A, C, Z = case.oracle()
    got, got_lse = attend(case)
    check_attention(got, got_lse, (out, lse, A, C, Z))


@BOTH
def test_visible_positions_without_a_page_are_skipped_and_reported(shape):
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(6, *shape)
    case.table[0, 0], case.table[0, 3], case.table[2, 4] = -1, case.pages, 2 ** 31 - 1
    case.table[1, :] = -5                                    # a request that has no page at all
    got, lse = attend(case, check=False)
    check_attention(got, lse, case.oracle())
    rows = slice(case.starts[1], case.starts[2])
    assert np.all(got[rows] == 0.0) and np.all(np.isneginf(lse[rows]))
    with pytest.raises(dsa.DsaError, match="BAD_PAGE"):
        attend(case)


@pytest.mark.parametrize("shape", [([700, 300], [1, 2], 32, 2, 8), ([700, 300], [20, 30], 32, 2, 8)], ids=["decode", "prompt"])
@pytest.mark.parametrize("gone", ["first", "last", "middle"])
def test_whole_tiles_without_a_page_before_keys_that_score_low(shape, gone):
    case = Kv4Case(20, *shape)
    P = case.P
    lo, hi = {"first": (0, 256), "last": (384, 700), "middle": (128, 640)}[gone]
    case.table[0, -(-lo // P):hi // P + 1] = -1
    case.table[1, :4] = -1
    slopes = np.full(case.heads, 2.0, np.float32)            # keys 100 away score -200 and less
    got, lse = attend(case, check=False, slopes=slopes)
    check_attention(got, lse, case.oracle(slopes=slopes), reach=2.0 * 700)


@BOTH
def test_a_request_longer_than_its_table_row_is_read_as_far_as_it_goes(shape):
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(7, *shape, extra_width=0)
    cache, batch, q = case.gpu()
    batch.seq_lens[0] = 50000
    with pytest.raises(dsa.DsaError, match="BAD_PAGE"):
        attend(case, (cache, batch, q))
    got, lse = attend(case, (cache, batch, q), check=False)
    want = [np.array(x) for x in case.oracle()]
    want[4][:case.starts[1]] = np.nan
    check_attention(got, lse, want)


def test_a_request_with_more_rows_than_announced_is_left_alone():
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(8, [300, 77, 129], [2, 30, 1], 32, 2, 8, extra_rows=2)
    with pytest.raises(dsa.DsaError, match="BAD_LENGTH"):
        attend(case, longest=4)
    got, lse = attend(case, longest=4, check=False)
    want = [np.array(x) for x in case.oracle()]
    want[4][2:32] = np.nan
    check_attention(got, lse, want)
    assert np.all(got[2:32] == -7.0) and np.all(lse[2:32] == -7.0)
    assert np.all(got[33:] == -7.0) and np.all(lse[33:] == -7.0)


@pytest.mark.parametrize("n", range(2))
def test_rows_that_come_before_the_sequence_see_nothing(n):
    """More rows than tokens: the first rows have no position."""
    case = Kv4Case(9, [5, 0, 40], [(9, 7, 1), (40, 33, 41)][n], 16, 1, 6, extra_rows=1)
    got, lse = attend(case)
    check_attention(got, lse, case.oracle())
    assert np.all(got[-1] == -7.0) and np.all(lse[-1] == -7.0)
    prefix = np.array([3, 2, 50], np.int32)
    got, lse = attend(case, prefix_lens=prefix)
    check_attention(got, lse, case.oracle(prefix=prefix))


@pytest.mark.parametrize("shape", [([20000, 9000], [1, 2], 64, 1, 8), ([3000, 40, 2600, 1500], [1, 1, 4, 1], 16, 2, 5),
                                   ([4100, 2500], [9, 70], 64, 1, 8), ([2100, 1500, 900], [100, 1, 40], 128, 2, 16),
                                   ([2400], [5], 32, 2, 64)])
@pytest.mark.parametrize("mods", [False, True])
def test_requests_that_many_ctas_share(shape, mods):
    case = Kv4Case(10, *shape)
    kw = {}
    if mods:
        kw = dict(softcap=3.0, slopes=case.slopes, prefix_lens=np.array([L // 2 for L in shape[0]], np.int32))
    got, lse = attend(case, **kw)
    if mods:
        kw["prefix"] = kw.pop("prefix_lens")
    check_attention(got, lse, case.oracle(**kw), softcap=3.0 if mods else 0.0, reach=float(case.slopes.max()) * max(shape[0]) if mods else 0.0)


@pytest.mark.parametrize("B,hi,group", [(700, 40, 2), (4096, 3, 1), (300, 1300, 4)])
def test_many_requests(B, hi, group):
    rng = np.random.default_rng(B)
    seq = rng.integers(0, hi + 1, B)
    new = np.minimum(seq, rng.integers(0, 3, B))
    new[-1] = min(seq[-1], 1)
    case = Kv4Case(11, seq.tolist(), new.tolist(), 16, 1, group)
    got, lse = attend(case)
    check_attention(got, lse, case.oracle())


@pytest.mark.parametrize("many", [False, True])
def test_the_most_requests_with_the_most_columns(many):
    rng = np.random.default_rng(42)
    seq = np.where(rng.random(4096) < 0.05, rng.integers(1, 200, 4096), 0)
    new = np.minimum(seq, rng.integers(1, 3, 4096))
    if many:
        new[[17, 4000]] = seq[[17, 4000]] = 9, 30
    case = Kv4Case(42, seq.tolist(), new.tolist(), 16, 1, 32)
    got, lse = attend(case)
    check_attention(got, lse, case.oracle())


def test_many_requests_of_many_rows():
    rng = np.random.default_rng(12)
    new = rng.integers(0, 23, 150)
    seq = new + rng.integers(0, 200, 150)
    seq[149] = 1400                                          # long enough that pieces are joined
    case = Kv4Case(12, seq.tolist(), new.tolist(), 16, 1, 8)
    got, lse = attend(case)
    check_attention(got, lse, case.oracle())


@pytest.mark.parametrize("seed", range(16))
def test_drawn_batches(seed):
    rng = np.random.default_rng(2000 + seed)
    B, P, kv = int(rng.integers(1, 9)), int(rng.choice([16, 32, 64, 128])), int(rng.integers(1, 4))
    group = int(rng.integers(1, 20))
    new = np.where(rng.random(B) < 0.5, rng.integers(0, 6, B), rng.integers(1, 60, B))
    seq = new + rng.integers(0, int(rng.choice([10, 400, 1500])), B)
    case = Kv4Case(2100 + seed, seq.tolist(), new.tolist(), P, kv, group, extra_rows=1 + int(rng.integers(0, 3)), spread=float(rng.random() * 3))
    kw = {}
    if rng.random() < 0.4:
        kw["softcap"] = float(rng.choice([0.5, 4.0, 30.0]))
    if rng.random() < 0.4:
        kw["slopes"] = case.slopes
    if rng.random() < 0.4:
        kw["prefix_lens"] = rng.integers(-2, 200, B).astype(np.int32)
    scale = float(rng.choice([128 ** -0.5, 0.02, 0.3]))
    got, lse = attend(case, scale=scale, **kw)
    if "prefix_lens" in kw:
        kw["prefix"] = kw.pop("prefix_lens")
    reach = float(case.slopes.max()) * float(seq.max()) if "slopes" in kw else 0.0
    check_attention(got, lse, case.oracle(scale=scale, **kw), softcap=kw.get("softcap", 0.0), reach=reach)


@BOTH
@pytest.mark.parametrize("cap", [1e-3, 63.0, 65.0, 1e6, 1e30])
def test_caps_of_any_size(shape, cap):
    """The bound does not grow with a large cap: scores are held to their own rounding."""
    case = Kv4Case(34, *shape)
    got, lse = attend(case, scale=0.5, softcap=cap)
    check_attention(got, lse, case.oracle(scale=0.5, softcap=cap))


@pytest.mark.parametrize("rows", [1, 3, 8, 20])
@pytest.mark.parametrize("before", [1 << 24, 1 << 25])
def test_a_distance_bias_past_two_to_the_24_tokens(rows, before):
    """Keys further than 1,000 away weigh e^-500 and less: one page stands for all of them."""
    import deepseek_sparse_mla_gb300 as dsa
    import torch
    case = Kv4Case(36, [1001], [rows], 128, 1, 8)
    filler = int(np.setdiff1d(np.arange(case.pages), case.table[0])[0])
    case.cache["k"][filler], case.cache["v"][filler], case.cache["ks"][filler], case.cache["vs"][filler] = 0, 0, 127, 1.0
    slopes = np.full(case.heads, 0.5, np.float32)
    want = case.oracle(slopes=slopes)
    cache, batch, q = case.gpu()
    table = torch.full((1, before // 128 + 8), filler, dtype=torch.int32, device="cuda")
    table[0, before // 128:] = batch.block_table[0, :8]
    far = dsa.Batch(table, batch.seq_lens + before, batch.query_start_loc, num_rows=rows, max_seq_len=before + 1001)
    got, lse = attend(case, (cache, far, q), slopes=slopes)
    check_attention(got, lse, want, reach=0.5 * 64)


@BOTH
def test_queries_of_a_fused_projection_and_no_lse(shape):
    import torch
    case = Kv4Case(13, *shape)
    cache, batch, q = case.gpu()
    wide = torch.full((case.rows, case.heads + 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + case.heads] = q
    got, _ = attend(case, (cache, batch, wide[:, 2:2 + case.heads]), want_lse=False)
    base, _ = attend(case, (cache, batch, q))
    assert np.array_equal(got, base)
    check_attention(got, None, case.oracle())


def test_decode_without_row_offsets():
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(14, [300, 0, 5], [1, 1, 1], 64, 2, 4)
    cache, batch, q = case.gpu()
    plain = dsa.Batch(batch.block_table, batch.seq_lens, None, num_rows=3, max_seq_len=300)
    got, lse = attend(case, (cache, plain, q))
    check_attention(got, lse, case.oracle())


@pytest.mark.parametrize("shape", [([2300, 77, 129], [1, 3, 2], 32, 2, 8), ([2300, 77, 129], [45, 9, 129], 32, 2, 8)],
                         ids=["decode", "prompt"])
def test_results_do_not_depend_on_the_workspace_the_stream_or_the_call(shape):
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(15, *shape)
    tensors = case.gpu()
    base, base_lse = attend(case, tensors)
    check_attention(base, base_lse, case.oracle())
    size = dsa.paged_attention_workspace_bytes(case.heads, case.kv, int(case.q_lens.max()))
    for fill in (0xFF, 0x00, 0x7F):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            got, lse = attend(case, tensors, workspace=ws)
            assert np.array_equal(got, base) and np.array_equal(lse, base_lse)
    side = torch.cuda.Stream()
    cache, batch, q = tensors
    out = [torch.zeros((case.rows, case.heads, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    dsa.paged_attention(cache, batch, q, max_query_len=int(case.q_lens.max()), out=out[0], stream=side)   # two calls at once
    dsa.paged_attention(cache, batch, q, max_query_len=int(case.q_lens.max()), out=out[1])
    torch.cuda.synchronize()
    for t in out:
        assert np.array_equal(o.bf16_to_f64(wlm.torch_to_bits(t)), base)


@pytest.mark.parametrize("group", [1, 5, 6, 20, 24])
def test_equal_calls_give_equal_bits_whatever_ran_between_them(group):
    """Columns and rows that no query or key fills keep what an earlier call left in shared memory: they do not count."""
    case = Kv4Case(37, [2300, 1800, 2777, 900] * 10, [1] * 40, 64, 2, group)
    wide = 8 if group <= 8 else 32
    others = [Kv4Case(38, [2500] * 40, [1] * 40, 64, 2, wide), Kv4Case(39, [700] * 40, [1] * 40, 64, 2, wide)]
    for c, up in zip(others, (64.0, 2.0 ** -20)):
        c.q_bits = wlm.bf16_bits((c.q * up).astype(np.float32))
    others[1].cache["ks"][:], others[1].cache["vs"][:] = f.NAN_SCALE, np.nan
    tensors, busy = case.gpu(), [c.gpu() for c in others]
    first = None
    for between in (None, 0, 1, 0, None):
        if between is not None:
            attend(others[between], busy[between])
        got = attend(case, tensors)
        first = first or got
        assert np.array_equal(got[0], first[0]) and np.array_equal(got[1], first[1]), f"after {between}"
    check_attention(*first, case.oracle())


@pytest.mark.parametrize("shape", [([1800, 77], [1, 3], 32, 2, 8), ([1800, 77], [45, 9], 32, 2, 8)], ids=["decode", "prompt"])
def test_two_captured_calls_replayed_over_changing_inputs(shape):
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    cases = [Kv4Case(16 + i, *shape) for i in range(2)]
    longest = int(cases[0].q_lens.max())
    tensors = [c.gpu() for c in cases]
    graphs, outs = [], []
    for c, (cache, batch, q) in zip(cases, tensors):
        ws = torch.empty(dsa.paged_attention_workspace_bytes(c.heads, c.kv, longest), dtype=torch.uint8, device="cuda")
        out = torch.zeros((c.rows, c.heads, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((c.rows, c.heads), dtype=torch.float32, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dsa.paged_attention(cache, batch, q, max_query_len=longest, out=out, lse=lse, workspace=ws)
        graphs.append((g, ws))
        outs.append((out, lse))
    for swap in range(3):
        for out, lse in outs:
            out.zero_(), lse.zero_()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, (out, lse) in zip(cases, outs):
            check_attention(o.bf16_to_f64(wlm.torch_to_bits(out)), lse.cpu().numpy().astype(np.float64), c.oracle())
        rng = np.random.default_rng(swap)
        for c, (_, batch, q) in zip(cases, tensors):         # shorter requests and other queries in place
            c.seq_lens = np.maximum(c.seq_lens - rng.integers(0, 300, c.seq_lens.shape), c.q_lens).astype(np.int32)
            batch.seq_lens.copy_(put(c.seq_lens))
            c.q_bits = wlm.bf16_bits(rng.standard_normal(c.q_bits.shape).astype(np.float32))
            q.copy_(wlm.bits_to_torch(c.q_bits, "cuda"))


def test_calls_over_both_caches_in_a_row_share_a_workspace():
    """Few-row and many-row requests whose pieces are joined, call after call without a wait in between."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    from dense_cases import DenseCase
    cases = [kind(22 + i, seq, new, 32, 2, 8) for i, (kind, seq, new) in enumerate(
        [(Kv4Case, [2300, 77, 1500], [1, 3, 60]), (DenseCase, [1200, 1900], [40, 2]), (Kv4Case, [1700], [1]), (Kv4Case, [1500], [70])])]
    tensors = [c.gpu() for c in cases]
    ws = torch.empty(dsa.paged_attention_workspace_bytes(16, 2, 70), dtype=torch.uint8, device="cuda")
    outs = []
    torch.cuda.synchronize()
    for turn in range(12):
        for c, (cache, batch, q) in zip(cases, tensors):
            out = torch.full((c.rows, c.heads, 128), -7.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.full((c.rows, c.heads), -7.0, dtype=torch.float32, device="cuda")
            dsa.paged_attention(cache, batch, q, max_query_len=int(c.q_lens.max()), out=out, lse=lse, workspace=ws)
            outs.append((out, lse))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(outs):
        first = outs[i % len(cases)]
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    for c, (out, lse) in zip(cases, outs):
        check_attention(o.bf16_to_f64(wlm.torch_to_bits(out)), lse.cpu().numpy().astype(np.float64), c.oracle())


@BOTH
def test_pages_past_four_gigabytes(shape):
    """The case's pages at the end of a cache of more than 2^32 bytes of K and of V."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(18, *shape)
    pages = (1 << 32) // (case.kv * case.P * 64) + 1000
    assert pages * case.kv * case.P < 2 ** 31
    first = pages - case.pages
    cache, batch, q = case.gpu()
    big = []
    for small, fill in ((cache.k_codes, 0x77), (cache.v_codes, 0x77), (cache.k_scales, 255), (cache.v_scales, float("nan"))):
        t = torch.full((pages, *small.shape[1:]), fill, dtype=small.dtype, device="cuda")
        t[first:] = small
        big.append(t)
    table = torch.where(batch.block_table >= 0, batch.block_table + first, batch.block_table)
    far = dsa.Kv4Cache.of(*big)
    b = dsa.Batch(table, batch.seq_lens, batch.query_start_loc, num_rows=case.rows, max_seq_len=300)
    got, lse = attend(case, (far, b, q))
    check_attention(got, lse, case.oracle())
    new = {n: wlm.bits_to_torch(case.new[n], "cuda") for n in "kv"}
    rope = dsa.RotaryTable.of(put(rope_table(300, 64)))
    dsa.kv4_append(cache, batch, new["k"], new["v"], rope=rope)
    dsa.kv4_append(far, b, new["k"], new["v"], rope=rope)
    torch.cuda.synchronize()
    for t, c in ((far.k_codes, cache.k_codes), (far.v_codes, cache.v_codes), (far.k_scales, cache.k_scales),
                 (far.v_scales.view(torch.int16), cache.v_scales.view(torch.int16))):
        assert torch.equal(t[first:], c)
        assert not torch.any(t[:first] != t[0]).item()


@pytest.mark.parametrize("new", [[3, 2, 4], [40, 30, 50]])
def test_offsets_that_run_back_or_leave_the_batch_are_reported(new):
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(43, [300, 77, 129], new, 32, 2, 8)
    cache, batch, q = case.gpu()
    end = int(case.starts[2])                                # the first two requests' rows
    want = [np.array(x) for x in case.oracle()]
    want[4][end:] = np.nan                                   # what is not compared
    for last in (end - 1, case.rows + 1, -5):
        batch.query_start_loc[3] = last
        with pytest.raises(dsa.DsaError, match="BAD_LENGTH"):
            attend(case, (cache, batch, q))
        got, lse = attend(case, (cache, batch, q), check=False)
        check_attention(got, lse, want)
        assert np.all(got[end:] == -7.0) and np.all(lse[end:] == -7.0)
    batch.query_start_loc.copy_(put(case.starts - 1))        # the first request's rows begin before the batch's
    with pytest.raises(dsa.DsaError, match="BAD_LENGTH"):
        attend(case, (cache, batch, q))


def test_calls_without_rows():
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(26, [50, 0], [0, 0], 16, 2, 2, extra_rows=1)
    cache, batch, q = case.gpu()
    got, lse = attend(case, (cache, batch, q), longest=40)   # a padded row only: it is left alone, and nothing is wrong
    assert np.all(got == -7.0) and np.all(lse == -7.0)
    none = dsa.Batch(batch.block_table, batch.seq_lens, batch.query_start_loc, num_rows=0, max_seq_len=50)
    out, _ = dsa.paged_attention(cache, none, q[:0], check=True)
    assert out.shape == (0, 4, 128)
    kv = wlm.bits_to_torch(case.new["k"], "cuda")[:0]
    before = cache.k_codes.clone()
    turned = dsa.kv4_append(cache, none, kv, kv, rope=dsa.RotaryTable(50, 64), q=q[:0])
    torch.cuda.synchronize()
    assert turned.shape == (0, 4, 128) and torch.equal(before, cache.k_codes)


def test_many_long_requests():
    """608 requests of 2^22 tokens, four to a CTA: segments and queries are ready requests ahead, and wait long for the next."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(44, [8192], [4], 128, 1, 8)
    cache, _, q = case.gpu()
    B, times = 608, 512
    table = put(np.tile(case.table[0, :64], times).astype(np.int32)).expand(B, 64 * times).contiguous()
    batch = dsa.Batch(table, put(np.full(B, 8192 * times, np.int32)), put(np.arange(B + 1, dtype=np.int32) * 4), num_rows=4 * B,
                      max_seq_len=8192 * times)
    lse = torch.zeros((4 * B, 8), dtype=torch.float32, device="cuda")
    out, _ = dsa.paged_attention(cache, batch, q.repeat(B, 1, 1), max_query_len=4, lse=lse, check=True)
    got, got_lse = o.bf16_to_f64(wlm.torch_to_bits(out)).reshape(B, 4, 8, 128), lse.cpu().numpy().astype(np.float64).reshape(B, 4, 8)
    pages, s = case.table[0, np.arange(8192) // 128], np.arange(8192) % 128
    k = f.values(case.cache["k"][pages, 0, s]) * np.repeat(np.exp2(case.cache["ks"][pages, 0, s].astype(np.float64) - 127), 32, -1)
    v = f.values(case.cache["v"][pages, 0, s]) * case.cache["vs"][pages, 0, s][:, None]
    z = np.einsum("kd,rhd->rhk", k, case.q) * 128 ** -0.5
    for i in range(4):
        w = np.exp(z[i]) * np.where(np.arange(8192) < 8192 - (3 - i), times, times - 1.0)
        total = w.sum(1)
        want, A = w @ v / total[:, None], w @ np.abs(v) / total[:, None]
        # two e4m3 terms of a contribution and bf16's half step, 2^-8 each, and the sums over 2^15 tiles
        assert np.all(np.abs(got[:, i] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * A + 2.0 ** -10)
        assert np.all(np.abs(got_lse[:, i] - np.log(total)) <= 2.0 ** -13 * 14)


def test_refusals():
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = Kv4Case(19, [50], [3], 16, 2, 2)
    cache, batch, q = case.gpu()
    k = wlm.bits_to_torch(case.new["k"], "cuda")
    for bad in (q.float(), q[:2], q[:, :, :64], q[0], q.cpu(), q.transpose(0, 1).contiguous().transpose(0, 1)[:, :0]):
        with pytest.raises((ValueError, dsa.DsaError)):
            dsa.paged_attention(cache, batch, bad, max_query_len=3)
    for bad in (k.float(), k[:, :1], k[:2], k.transpose(1, 2).contiguous().transpose(1, 2), k.cpu()):
        with pytest.raises(ValueError):
            dsa.kv4_append(cache, batch, bad, k)
    rope = dsa.RotaryTable(50, 64)
    with pytest.raises(ValueError, match="rope"):
        dsa.kv4_append(cache, batch, k, k, q=q)
    with pytest.raises(ValueError, match="q_out"):
        dsa.kv4_append(cache, batch, k, k, rope=rope, q_out=q)
    with pytest.raises(ValueError, match="q:"):
        dsa.kv4_append(cache, batch, k, k, rope=rope, q=q[:2])
    with pytest.raises(ValueError, match="q_out"):
        dsa.kv4_append(cache, batch, k, k, rope=rope, q=q, q_out=q[:, :2])
    with pytest.raises(dsa.DsaError, match="positions"):
        dsa.kv4_append(cache, batch, k, k, rope=dsa.RotaryTable(49, 64))
    with pytest.raises(dsa.DsaError, match="dim"):
        dsa.kv4_append(cache, batch, k, k, rope=dsa.RotaryTable(50, 48))
    with pytest.raises(ValueError, match="cos_sin"):
        dsa.RotaryTable.of(torch.zeros(50, 64, dtype=torch.bfloat16, device="cuda"))
    codes = torch.zeros(4, 2, 64, 64, dtype=torch.uint8, device="cuda")
    ks, vs = torch.zeros(4, 2, 64, 4, dtype=torch.uint8, device="cuda"), torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="v_codes"):
        dsa.Kv4Cache.of(codes, codes[:3], ks, vs)
    with pytest.raises(ValueError, match="k_scales"):
        dsa.Kv4Cache.of(codes, codes.clone(), ks.float(), vs)
    with pytest.raises(ValueError, match="v_scales"):
        dsa.Kv4Cache.of(codes, codes.clone(), ks, vs.float())
    shifted = torch.zeros(4 * 2 * 64 * 64 + 16, dtype=torch.uint8, device="cuda")[16:].view(4, 2, 64, 64)
    with pytest.raises(dsa.DsaError, match="32-byte"):
        dsa.paged_attention(dsa.Kv4Cache.of(shifted, codes, ks, vs), batch, q)
