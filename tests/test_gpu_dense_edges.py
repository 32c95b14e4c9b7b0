"""Dense attention on the GPU where it can go wrong: masked and visible NaN, wide scales, bad pages, rows that are left alone,
long and many requests, strides, streams, graphs and stale workspaces.  Every case runs in the kernel for few rows and, with
more than 64 rows * heads a request, in the one for prompts."""
import numpy as np
import pytest

import workloads as wlm
from dense_cases import DenseCase, check_attention
from oracle import dsa_oracle as o

pytestmark = pytest.mark.gpu

DECODE = ([300, 77, 129], [1, 3, 2], 32, 2, 8)
PROMPT = ([300, 77, 129], [45, 9, 129], 32, 2, 8)


def put(a):
    import torch
    return torch.from_numpy(np.array(a)).cuda()


def attend(case, tensors=None, longest=None, check=True, workspace=None, want_lse=True, scale=128 ** -0.5, **mods):
    """(out as float64, lse as float64) with rows that no kernel wrote at -7."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    cache, batch, q = tensors or case.gpu()
    out = torch.full((case.rows, case.heads, 128), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.rows, case.heads), -7.0, dtype=torch.float32, device="cuda") if want_lse else None
    mods = {k: put(v) if isinstance(v, np.ndarray) else v for k, v in mods.items()}
    dsa.paged_attention(cache, batch, q, scale, max_query_len=longest or max(1, int(case.q_lens.max())), out=out, lse=lse,
                        workspace=workspace, check=check, **mods)
    torch.cuda.synchronize()
    return o.bf16_to_f64(wlm.torch_to_bits(out)), None if lse is None else lse.cpu().numpy().astype(np.float64)


def row_limits(case):
    """Keys seen by each row, and each row's request."""
    limit, req = np.zeros(case.rows, np.int64), np.full(case.rows, -1)
    for b, L in enumerate(case.seq_lens):
        n = case.q_lens[b]
        limit[case.starts[b]:case.starts[b + 1]] = L - n + 1 + np.arange(n)
        req[case.starts[b]:case.starts[b + 1]] = b
    return limit, req


@pytest.mark.parametrize("shape", [DECODE, PROMPT], ids=["decode", "prompt"])
def test_a_nan_in_v_reaches_its_dim_of_the_rows_that_see_it(shape):
    case = DenseCase(1, *shape)
    want = [np.array(x) for x in case.oracle()]
    limit, req = row_limits(case)
    out = want[0]
    for b, key, h, dim in ((0, 12, 1, 5), (0, 298, 0, 127), (1, 76, 0, 64), (2, 127, 1, 0), (2, 128, 1, 1)):
        case.codes["v"][case.table[b, key // case.P], h, key % case.P, dim] = 0xFF if dim & 1 else 0x7F
        rows = (req == b) & (limit > key)
        out[rows, h * case.group:(h + 1) * case.group, dim] = np.nan
    got, lse = attend(case)
    nan = np.isnan(out)
    assert np.array_equal(np.isnan(got), nan)
    clean = [np.where(nan, 0.0, out), want[1], *want[2:]]
    check_attention(np.where(nan, 0.0, got), lse, clean)


@pytest.mark.parametrize("shape", [DECODE, PROMPT], ids=["decode", "prompt"])
def test_a_nan_in_k_reaches_the_rows_that_see_it(shape):
    case = DenseCase(2, *shape)
    want = [np.array(x) for x in case.oracle()]
    limit, req = row_limits(case)
    bad = np.zeros((case.rows, case.heads), bool)
    for b, key, h in ((0, 299, 1), (1, 74, 0), (2, 100, 1)):
        case.codes["k"][case.table[b, key // case.P], h, key % case.P, 17] = 0x7F
        bad[np.ix_((req == b) & (limit > key), range(h * case.group, (h + 1) * case.group))] = True
    got, lse = attend(case)
    assert np.array_equal(np.isnan(lse), bad) and np.array_equal(np.isnan(got), np.broadcast_to(bad[..., None], got.shape))
    want[4] = np.where(bad, np.nan, want[4])                 # what the check leaves out
    check_attention(got, np.where(bad, 0.0, lse), want)


@pytest.mark.parametrize("shape", [DECODE, PROMPT], ids=["decode", "prompt"])
def test_a_query_that_is_not_finite_poisons_its_own_pair_only(shape):
    case = DenseCase(3, *shape)
    want = [np.array(x) for x in case.oracle()]
    bad = np.zeros((case.rows, case.heads), bool)
    for r, h, bits in ((0, 3, 0x7FC0), (2, 15, 0x7F80), (case.rows - 1, 0, 0xFF80)):
        case.q_bits[r, h, 9] = bits
        bad[r, h] = True
    got, lse = attend(case)
    assert np.array_equal(np.isnan(lse), bad) and np.array_equal(np.isnan(got), np.broadcast_to(bad[..., None], got.shape))
    want[4] = np.where(bad, np.nan, want[4])
    check_attention(got, np.where(bad, 0.0, lse), want)


@pytest.mark.parametrize("shape", [DECODE, PROMPT], ids=["decode", "prompt"])
def test_page_scales_far_apart_and_of_zero(shape):
    case = DenseCase(4, *shape)
    rng = np.random.default_rng(4)
    case.scales["v"] *= np.exp2(rng.integers(-24, 25, case.scales["v"].shape)).astype(np.float32)
    case.scales["k"] *= np.exp2(rng.integers(-24, 1, case.scales["k"].shape)).astype(np.float32)
    case.scales["v"][case.table[0, 1]] = 0.0
    case.scales["k"][case.table[0, 2]] = 0.0
    case.scales["v"][case.table[1, :3], 1] = 0.0             # a request and head whose values are all zero
    got, lse = attend(case)
    want = case.oracle()
    check_attention(got, lse, want)
    rows = slice(case.starts[1], case.starts[2])
    assert np.all(got[rows, case.group:] == 0.0)


@pytest.mark.parametrize("shape", [DECODE, PROMPT], ids=["decode", "prompt"])
def test_the_smallest_and_largest_scales(shape):
    case = DenseCase(5, *shape)
    case.scales["k"][:] = 2.0 ** -126
    case.scales["v"][:] = 2.0 ** -126
    got, lse = attend(case)                                  # outputs of a few 2^-126: what bf16 has no normal number for is 0
    assert np.all(np.abs(got[:int(case.starts[-1])]) < 2.0 ** -115)
    case.scales["v"][:] = 2.0 ** 110
    got, lse = attend(case)
    check_attention(got, lse, case.oracle())


def test_the_scale_of_a_page_that_only_later_rows_see_leaves_the_others_alone():
    case = DenseCase(21, [65, 131], [3, 4], 16, 2, 8)
    for name in "kv":
        case.scales[name][case.table[0, :4]] *= np.float32(2.0 ** -30)
        case.scales[name][case.table[1, :8]] *= np.float32(2.0 ** -30)
    case.scales["v"][case.table[0, 4]] = 2.0 ** 118          # the last row's own page
    case.scales["v"][case.table[1, 8]] = 2.0 ** 118
    got, lse = attend(case)
    check_attention(got, lse, case.oracle())


@pytest.mark.parametrize("shape", [DECODE, PROMPT], ids=["decode", "prompt"])
def test_visible_positions_without_a_page_are_skipped_and_reported(shape):
    import deepseek_sparse_mla_gb300 as dsa
    case = DenseCase(6, *shape)
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
    case = DenseCase(20, *shape)
    P = case.P
    lo, hi = {"first": (0, 256), "last": (384, 700), "middle": (128, 640)}[gone]
    case.table[0, -(-lo // P):hi // P + 1] = -1
    case.table[1, :4] = -1
    slopes = np.full(case.heads, 2.0, np.float32)            # keys 100 away score -200 and less
    got, lse = attend(case, check=False, slopes=slopes)
    check_attention(got, lse, case.oracle(slopes=slopes), reach=2.0 * 700)


@pytest.mark.parametrize("shape", [DECODE, PROMPT], ids=["decode", "prompt"])
def test_a_request_longer_than_its_table_row_is_read_as_far_as_it_goes(shape):
    import deepseek_sparse_mla_gb300 as dsa
    case = DenseCase(7, *shape, extra_width=0)
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
    case = DenseCase(8, [300, 77, 129], [2, 30, 1], 32, 2, 8, extra_rows=2)
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
    case = DenseCase(9, [5, 0, 40], [(9, 7, 1), (40, 33, 41)][n], 16, 1, 6, extra_rows=1)
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
    case = DenseCase(10, *shape)
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
    case = DenseCase(11, seq.tolist(), new.tolist(), 16, 1, group)
    got, lse = attend(case)
    check_attention(got, lse, case.oracle())


def test_many_requests_of_many_rows():
    rng = np.random.default_rng(12)
    new = rng.integers(0, 23, 150)
    seq = new + rng.integers(0, 200, 150)
    seq[149] = 1400                                          # long enough that pieces are joined
    case = DenseCase(12, seq.tolist(), new.tolist(), 16, 1, 8)
    got, lse = attend(case)
    check_attention(got, lse, case.oracle())


@pytest.mark.parametrize("seed", range(16))
def test_drawn_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    B, P, kv = int(rng.integers(1, 9)), int(rng.choice([16, 32, 64, 128])), int(rng.integers(1, 4))
    group = int(rng.integers(1, 20))
    new = np.where(rng.random(B) < 0.5, rng.integers(0, 6, B), rng.integers(1, 60, B))
    seq = new + rng.integers(0, int(rng.choice([10, 400, 1500])), B)
    case = DenseCase(1100 + seed, seq.tolist(), new.tolist(), P, kv, group, extra_rows=int(rng.integers(0, 3)), spread=float(rng.random() * 3))
    if case.rows == 0:
        case = DenseCase(1100 + seed, seq.tolist(), new.tolist(), P, kv, group, extra_rows=1)
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


@pytest.mark.parametrize("shape", [DECODE, PROMPT], ids=["decode", "prompt"])
def test_queries_of_a_fused_projection_and_no_lse(shape):
    import torch
    case = DenseCase(13, *shape)
    cache, batch, q = case.gpu()
    wide = torch.full((case.rows, case.heads + 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + case.heads] = q
    got, _ = attend(case, (cache, batch, wide[:, 2:2 + case.heads]), want_lse=False)
    base, _ = attend(case, (cache, batch, q))
    assert np.array_equal(got, base)
    check_attention(got, None, case.oracle())


def test_decode_without_row_offsets():
    import deepseek_sparse_mla_gb300 as dsa
    case = DenseCase(14, [300, 0, 5], [1, 1, 1], 64, 2, 4)
    cache, batch, q = case.gpu()
    plain = dsa.Batch(batch.block_table, batch.seq_lens, None, num_rows=3, max_seq_len=300)
    got, lse = attend(case, (cache, plain, q))
    check_attention(got, lse, case.oracle())


@pytest.mark.parametrize("shape", [([2300, 77, 129], [1, 3, 2], 32, 2, 8), ([2300, 77, 129], [45, 9, 129], 32, 2, 8)],
                         ids=["decode", "prompt"])
def test_results_do_not_depend_on_the_workspace_the_stream_or_the_call(shape):
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = DenseCase(15, *shape)
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


@pytest.mark.parametrize("shape", [([1800, 77], [1, 3], 32, 2, 8), ([1800, 77], [45, 9], 32, 2, 8)], ids=["decode", "prompt"])
def test_two_captured_calls_replayed_over_changing_inputs(shape):
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    cases = [DenseCase(16 + i, *shape) for i in range(2)]
    longest = int(cases[0].q_lens.max())
    # the second case's pool in the first one's tensors, so that a replay can switch
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


def test_calls_in_a_row_share_a_workspace():
    """Few-row and many-row requests whose pieces are joined, call after call without a wait in between."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    cases = [DenseCase(22 + i, seq, new, 32, 2, 8) for i, (seq, new) in enumerate(
        [([2300, 77, 1500], [1, 3, 60]), ([1200, 1900], [40, 2]), ([1700], [1]), ([1500], [70])])]
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


@pytest.mark.parametrize("shape", [DECODE, PROMPT], ids=["decode", "prompt"])
def test_pages_past_four_gigabytes(shape):
    """The case's pages at the end of a cache of more than 2^32 bytes of K and of V."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = DenseCase(18, *shape)
    pages = (1 << 32) // (case.kv * case.P * 128) + 1000
    first = pages - case.pages
    cache, batch, q = case.gpu()
    big = []
    for small in (cache.k_codes, cache.v_codes):
        t = torch.full((pages, case.kv, case.P, 128), 0x7F, dtype=torch.uint8, device="cuda")
        t[first:] = small
        big.append(t)
    for small in (cache.k_scales, cache.v_scales):
        t = torch.ones((pages, case.kv), dtype=torch.float32, device="cuda")
        t[first:] = small
        big.append(t)
    table = torch.where(batch.block_table >= 0, batch.block_table + first, batch.block_table)
    far = dsa.BlockKvCache.of(*big)
    b = dsa.Batch(table, batch.seq_lens, batch.query_start_loc, num_rows=case.rows, max_seq_len=300)
    got, lse = attend(case, (far, b, q))
    check_attention(got, lse, case.oracle())
    new = {n: wlm.bits_to_torch(case.new[n], "cuda") for n in "kv"}
    dsa.kv8_append(cache, batch, new["k"], new["v"])
    dsa.kv8_append(far, b, new["k"], new["v"])
    torch.cuda.synchronize()
    for a, c in ((far.k_codes, cache.k_codes), (far.v_codes, cache.v_codes), (far.k_scales, cache.k_scales), (far.v_scales, cache.v_scales)):
        assert torch.equal(a[first:], c)
        assert not torch.any(a[:first] != a[0]).item()


def test_calls_without_rows():
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = DenseCase(26, [50, 0], [0, 0], 16, 2, 2, extra_rows=1)
    cache, batch, q = case.gpu()
    got, lse = attend(case, (cache, batch, q), longest=40)   # a padded row only: it is left alone, and nothing is wrong
    assert np.all(got == -7.0) and np.all(lse == -7.0)
    none = dsa.Batch(batch.block_table, batch.seq_lens, batch.query_start_loc, num_rows=0, max_seq_len=50)
    ws = torch.full((dsa.paged_attention_workspace_bytes(4, 2, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    out, _ = dsa.paged_attention(cache, none, q[:0], workspace=ws, check=True)
    assert out.shape == (0, 4, 128)
    kv = wlm.bits_to_torch(case.new["k"], "cuda")[:0]
    before = cache.k_codes.clone()
    dsa.kv8_append(cache, none, kv, kv)
    torch.cuda.synchronize()
    assert torch.equal(before, cache.k_codes)


def test_refusals():
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = DenseCase(19, [50], [3], 16, 2, 2)
    cache, batch, q = case.gpu()
    for bad in (q.float(), q[:2], q[:, :, :64], q[0], q.cpu(), q.transpose(0, 1).contiguous().transpose(0, 1)[:, :0]):
        with pytest.raises((ValueError, dsa.DsaError)):
            dsa.paged_attention(cache, batch, bad, max_query_len=3)
    with pytest.raises(ValueError, match="slopes"):
        dsa.paged_attention(cache, batch, q, slopes=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError, match="prefix_lens"):
        dsa.paged_attention(cache, batch, q, prefix_lens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        dsa.paged_attention(cache, batch, q, out=torch.zeros_like(q)[:2])
    with pytest.raises(ValueError, match="lse"):
        dsa.paged_attention(cache, batch, q, lse=torch.zeros(3, 4, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(dsa.DsaError, match="softcap"):
        dsa.paged_attention(cache, batch, q, softcap=-1.0)
    with pytest.raises(dsa.DsaError, match="workspace"):
        dsa.paged_attention(cache, batch, q, workspace=torch.zeros(512, dtype=torch.uint8, device="cuda"))
    codes = torch.zeros(4, 2, 64, 128, dtype=torch.uint8, device="cuda")
    ones = torch.ones(4, 2, device="cuda")
    with pytest.raises(ValueError, match="v_codes"):
        dsa.BlockKvCache.of(codes, codes[:3], ones, ones)
    with pytest.raises(ValueError, match="v_scales"):
        dsa.BlockKvCache.of(codes, codes.clone(), ones, torch.ones(4, 3, device="cuda"))
