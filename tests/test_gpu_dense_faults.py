"""Dense attention on the GPU: inputs that were once answered wrongly, in both kernels."""
import numpy as np
import pytest

import workloads as wlm
from dense_cases import DenseCase, check_attention
from oracle import dsa_oracle as o

pytestmark = pytest.mark.gpu


def put(a):
    import torch
    return torch.from_numpy(np.array(a)).cuda()


def attend(case, tensors=None, longest=None, check=True, scale=128 ** -0.5, **mods):
    """(out as float64, lse as float64) with rows that no kernel wrote at -7."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    cache, batch, q = tensors or case.gpu()
    out = torch.full((case.rows, case.heads, 128), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.rows, case.heads), -7.0, dtype=torch.float32, device="cuda")
    mods = {k: put(v) if isinstance(v, np.ndarray) else v for k, v in mods.items()}
    dsa.paged_attention(cache, batch, q, scale, max_query_len=longest or max(1, int(case.q_lens.max())), out=out, lse=lse,
                        check=check, **mods)
    torch.cuda.synchronize()
    return o.bf16_to_f64(wlm.torch_to_bits(out)), lse.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("B,stride", [(64, 40), (4096, 8192)])
def test_starts_that_run_back_are_refused(B, stride):
    """Every other request names the same 2,048 rows of 16 heads: 128 groups of 256 pairs each time.  With 2,048 of them and
    8,192 tiles of 128 keys a group, the sum of the tiles would be 2^31."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    rows, P = 2048, 128
    starts = np.zeros(B + 1, np.int32)
    starts[1::2] = rows
    cache = dsa.BlockKvCache(4, P, 1)
    table = torch.zeros((B, stride), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), stride * P, dtype=torch.int32, device="cuda")
    batch = dsa.Batch(table, lens, put(starts), num_rows=rows, max_seq_len=stride * P)
    q = torch.zeros((rows, 16, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.full((rows, 16, 128), -7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dsa.DsaError, match="BAD_LENGTH"):
        dsa.paged_attention(cache, batch, q, max_query_len=rows, out=out, check=True)
    assert torch.all(out == -7.0).item()


@pytest.mark.parametrize("group", [1, 5, 6, 20, 24])
def test_equal_calls_give_equal_bits_whatever_ran_between_them(group):
    """Columns of a tile that no query fills keep what an earlier call left in shared memory: they do not count."""
    case = DenseCase(37, [2300, 1800, 2777, 900] * 10, [1] * 40, 64, 2, group)
    wide = 8 if group <= 8 else 32
    others = [DenseCase(38, [2500] * 40, [1] * 40, 64, 2, wide), DenseCase(39, [700] * 40, [1] * 40, 64, 2, wide)]
    for c, up in zip(others, (64.0, 2.0 ** -20)):
        c.q_bits = wlm.bf16_bits((c.q * up).astype(np.float32))
    tensors, busy = case.gpu(), [c.gpu() for c in others]
    first = None
    for between in (None, 0, 1, 0, None):
        if between is not None:
            attend(others[between], busy[between])
        got = attend(case, tensors)
        first = first or got
        same = np.array_equal(got[0], first[0]) and np.array_equal(got[1], first[1])
        assert same, f"after {between}"
    check_attention(*first, case.oracle())


def largest_contribution(case, lse, scale=128 ** -0.5):
    """max_s p_s |v_scale_s| * sum_s |v_code_s|, in the place of the oracle's C, which takes both maxima apart."""
    codes, C = {n: o.e4m3_to_f64(case.codes[n]) for n in "kv"}, np.zeros((case.rows, case.heads, 128))
    for b, L in enumerate(int(v) for v in case.seq_lens):
        at = np.arange(L)
        page, off = case.table[b, at // case.P], at % case.P
        for r in range(case.starts[b], case.starts[b + 1]):
            see = slice(0, L - case.q_lens[b] + 1 + r - case.starts[b])
            for head in range(case.heads):
                h = head // case.group
                k = codes["k"][page[see], h, off[see]] * case.scales["k"][page[see], h].astype(np.float64)[:, None]
                p = np.exp(scale * (k @ case.q[r, head]) - lse[r, head])
                vs = np.abs(case.scales["v"][page[see], h].astype(np.float64))
                C[r, head] = (p * vs).max() * np.abs(codes["v"][page[see], h, off[see]]).sum(0)
    return C


@pytest.mark.parametrize("seq,new", [([49], [3]), ([64, 81, 33], [5, 4, 2]), ([143, 17], [16, 2])])
def test_a_page_that_only_later_rows_see_leaves_the_others_their_bits(seq, new):
    """Pages of 16 tokens, two to a warp's 32 keys: the last one, with a scale far above the others', shares them with one that
    the earlier rows see."""
    case = DenseCase(31, seq, new, 16, 2, 4)
    for b, L in enumerate(seq):
        last = (L - 1) // 16
        case.scales["v"][case.table[b, :last]] *= np.float32(2.0 ** -30)
        case.scales["v"][case.table[b, last]] = 2.0 ** 118
    out, lse, A, _, Z = case.oracle()
    got, got_lse = attend(case)
    check_attention(got, got_lse, (out, lse, A, largest_contribution(case, lse), Z))


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("step", [3, 12])
@pytest.mark.parametrize("scale", [128 ** -0.5, 1.0])
def test_scales_far_apart_keep_the_bits_of_the_largest_contribution(P, step, scale):
    """Neighbouring pages whose scales of V, and with a scale of 1 whose scores too, lie far apart."""
    case = DenseCase(32, [300, 77, 129, 700], [1, 3, 2, 4], P, 2, 8)
    rng = np.random.default_rng(32)
    case.scales["v"] *= np.exp2(rng.integers(-2, 3, case.scales["v"].shape) * step).astype(np.float32)
    out, lse, A, _, Z = case.oracle(scale=scale)
    got, got_lse = attend(case, scale=scale)
    check_attention(got, got_lse, (out, lse, A, largest_contribution(case, lse, scale), Z))


SHAPES = {"decode": ([900, 77, 129], [1, 3, 2], 32, 2, 8), "prompt": ([900, 77, 129], [45, 9, 129], 32, 2, 8)}


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("cap", [24.0, 96.0, 1e3, 1e4, 1e6, 1e8, 1e12, 1e30])
def test_large_caps_leave_scores_as_they_are(shape, cap):
    """The bound does not grow with the cap: scores are held to their own rounding."""
    case = DenseCase(34, *SHAPES[shape])
    got, lse = attend(case, scale=0.5, softcap=cap)
    check_attention(got, lse, case.oracle(scale=0.5, softcap=cap))


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("cap", [1e-30, 1e-3, 0.1])
def test_small_caps(shape, cap):
    case = DenseCase(35, *SHAPES[shape])
    got, lse = attend(case, softcap=cap)
    check_attention(got, lse, case.oracle(softcap=cap))


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("cap", [63.0, 65.0, 1e5])
def test_a_large_cap_with_a_bias_and_a_prefix(shape, cap):
    case = DenseCase(40, *SHAPES[shape])
    prefix = np.array([200, 77, 10], np.int32)
    got, lse = attend(case, scale=0.5, softcap=cap, slopes=case.slopes, prefix_lens=prefix)
    want = case.oracle(scale=0.5, softcap=cap, slopes=case.slopes, prefix=prefix)
    check_attention(got, lse, want, reach=float(case.slopes.max()) * 900)


@pytest.mark.parametrize("rows", [1, 3, 8, 20])
@pytest.mark.parametrize("before", [1 << 24, 1 << 25])
def test_a_distance_bias_past_two_to_the_24_tokens(rows, before):
    """Keys further than 1,000 away weigh e^-500 and less: one page stands for all of them."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    case = DenseCase(36, [1001], [rows], 128, 1, 8)
    filler = int(np.setdiff1d(np.arange(case.pages), case.table[0])[0])
    for n in "kv":
        case.codes[n][filler] = 0
    slopes = np.full(case.heads, 0.5, np.float32)
    want = case.oracle(slopes=slopes)
    cache, batch, q = case.gpu()
    table = torch.full((1, before // 128 + 8), filler, dtype=torch.int32, device="cuda")
    table[0, before // 128:] = batch.block_table[0, :8]
    far = dsa.Batch(table, batch.seq_lens + before, batch.query_start_loc, num_rows=rows, max_seq_len=before + 1001)
    got, lse = attend(case, (cache, far, q), slopes=slopes)
    check_attention(got, lse, want, reach=0.5 * 64)


def test_a_prompts_values_are_held_to_a_share_of_the_requests_largest_scale():
    """The kernel for many rows holds V in half precision relative to the request's largest scale: half a step of its smallest
    numbers, 2^-25 of that scale, also for rows that do not see the page with it."""
    case = DenseCase(33, [600, 333], [40, 70], 16, 2, 8)
    tops = np.zeros((case.rows, 1, 1))
    for b, L in enumerate(case.seq_lens):
        last = case.table[b, (L - 1) // 16]
        case.scales["v"][last] *= np.float32(2.0 ** (14 + 4 * b))
        tops[case.starts[b]:case.starts[b + 1]] = case.scales["v"][case.table[b, :-(-L // 16)]].max()
    out, lse, A, C, Z = case.oracle()
    got, got_lse = attend(case)
    assert np.all(np.isfinite(got))
    dz = 2.0 ** -15 * Z + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -9 + 2 * dz[..., None]) * A + 2.0 ** -25 * tops   # bf16, P's 11 bits and the sums, V
    assert np.all(np.abs(got - out) <= tol)
    assert np.all(np.abs(got_lse - lse) <= dz + 2.0 ** -20 * (1 + np.abs(lse)))


FAR = {"decode": ([20000, 1100, 77], [1, 2, 2], 2, 8), "prompt": ([12000, 1100], [30, 45], 1, 8)}


@pytest.mark.parametrize("k", [-119, -110, -80, 80, 110, 125])
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("shape", list(FAR))
def test_values_of_any_size(shape, P, k):
    """V's scales from 2^-126 to 2^119, with pieces of long requests to join: the output is that of scales near one, times a power
    of two, up to the rounding of bf16's subnormal numbers."""
    seq, new, kv, group = FAR[shape]
    case = DenseCase(41, seq, new, P, kv, group, spread=0.0)
    out, lse, A, C, Z = case.oracle()
    assert np.abs(out).max() < 4.0 and case.scales["v"].min() >= 2.0 ** -7
    tensors = case.gpu()
    tensors[0].v_scales.copy_(put(np.ldexp(case.scales["v"], k).astype(np.float32)))
    got, got_lse = attend(case, tensors)
    C += 2.0 ** 18 * 2.0 ** (-134 - k)                       # half a step of those numbers (the bound takes 2^-18 of C)
    check_attention(np.ldexp(got, -k), got_lse, (out, lse, A, C, Z))


@pytest.mark.parametrize("many", [False, True])
def test_the_most_requests_with_the_most_columns(many):
    """The largest shared memory a call may ask for: 4,096 requests, most of them empty, and blocks of 32 columns."""
    rng = np.random.default_rng(42)
    seq = np.where(rng.random(4096) < 0.05, rng.integers(1, 200, 4096), 0)
    new = np.minimum(seq, rng.integers(1, 3, 4096))
    if many:
        new[[17, 4000]] = seq[[17, 4000]] = 9, 30
    case = DenseCase(42, seq.tolist(), new.tolist(), 16, 1, 32)
    got, lse = attend(case)
    check_attention(got, lse, case.oracle())


@pytest.mark.parametrize("new", [[3, 2, 4], [40, 30, 50]])
def test_offsets_that_run_back_or_leave_the_batch_are_reported(new):
    import deepseek_sparse_mla_gb300 as dsa
    case = DenseCase(43, [300, 77, 129], new, 32, 2, 8)
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


class Repeated:
    """64 pages of 128 tokens that long requests have over and over, queries, and what a row gets that sees all tokens of
    `times` rounds but the last `missing`."""

    def __init__(self, seed, rows):
        self.case = DenseCase(seed, [8192], [rows], 128, 1, 8, spread=0.5)
        pages = self.case.table[0, :64]
        self.k, self.v = ((o.e4m3_to_f64(self.case.codes[n][pages, 0]) * self.case.scales[n][pages, 0][:, None, None].astype(np.float64))
                          .reshape(-1, 128) for n in "kv")
        self.z = np.einsum("kd,rhd->rhk", self.k, self.case.q) * 128 ** -0.5

    def row(self, r, times, missing):
        w = np.exp(self.z[r]) * np.where(np.arange(8192) < 8192 - missing, times, times - 1.0)
        total = w.sum(1)
        return w @ self.v / total[:, None], np.log(total), w @ np.abs(self.v) / total[:, None]

    def run(self, kinds):
        """A call over requests of (count, rounds, rows); outputs and lse are checked for one of each kind, and all of a kind are
        equal up to the rounding of pieces and their sums."""
        import torch
        import deepseek_sparse_mla_gb300 as dsa
        cache, _, q = self.case.gpu()
        B, most, rows = sum(n for n, _, _ in kinds), max(t for _, t, _ in kinds), sum(n * r for n, _, r in kinds)
        table = put(np.tile(self.case.table[0, :64], (1, most)).astype(np.int32)).expand(B, 64 * most).contiguous()
        lens = np.concatenate([np.full(n, 8192 * t) for n, t, _ in kinds]).astype(np.int32)
        starts = np.concatenate([[0], np.cumsum(np.concatenate([np.full(n, r) for n, _, r in kinds]))]).astype(np.int32)
        batch = dsa.Batch(table, put(lens), put(starts), num_rows=rows, max_seq_len=8192 * most)
        q = torch.cat([q[:r].repeat(n, 1, 1) for n, _, r in kinds])
        lse = torch.zeros((rows, 8), dtype=torch.float32, device="cuda")
        out, _ = dsa.paged_attention(cache, batch, q, max_query_len=max(r for _, _, r in kinds), lse=lse, check=True)
        out, lse = o.bf16_to_f64(wlm.torch_to_bits(out)), lse.cpu().numpy().astype(np.float64)
        at = 0
        for n, t, r in kinds:
            got, got_lse = out[at:at + n * r].reshape(n, r, 8, 128), lse[at:at + n * r].reshape(n, r, 8)
            at += n * r
            for i in range(r):
                want, want_lse, A = self.row(i, float(t), r - 1 - i)
                # two e4m3 terms of a contribution and bf16's half step, 2^-8 each, and the sums over up to 2^15 tiles
                assert np.all(np.abs(got[:, i] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * A + 2.0 ** -10)
                assert np.all(np.abs(got_lse[:, i] - want_lse) <= 2.0 ** -13 * 14)


def test_many_long_requests():
    """608 requests of 2^22 tokens, four to a CTA: the queries are ready three requests ahead, and wait 57 ms for the next."""
    Repeated(44, 4).run([(608, 512, 4)])


def test_prompts_beside_long_requests_that_keep_some_ctas_longer():
    """Requests of one row and of eight have tiles of different cost: the first CTAs are done 10 ms and more before the last, and
    the prompts' kernel starts on their SMs, with more than one prompt each, before it may write."""
    Repeated(45, 16).run([(304, 64, 1), (76, 64, 8), (400, 1, 16)])
