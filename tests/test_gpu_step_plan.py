"""The step planner and the page release on the GPU against the oracle: whole numbers, equal."""
import numpy as np
import pytest

from oracle import dense_oracle as d

pytestmark = pytest.mark.gpu


def make(seed, B, P, hi, news, width=None, free=None, holes=False):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, hi + 1, B).astype(np.int32)
    new = np.array([news[i % len(news)] for i in range(B)], np.int32)
    rng.shuffle(new)
    held = -(-lens // P)
    need = -(-(lens.astype(np.int64) + np.maximum(new, 0)) // P) - held
    width = int(max(1, (held + need).max() + 1)) if width is None else width
    total = int(held.sum() + np.maximum(need, 0).sum()) + 5
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        n = min(width, int(held[b]))
        table[b, :n] = perm[at:at + n]
        at += n
    stack = np.full(total, -9, np.int32)
    count = total - at if free is None else free
    stack[:total - at] = perm[at:]
    return lens, new, table, stack, count, total


def plan(lens, new, table, stack, count, P, rows, check=False, in_place=False):
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    put = lambda a: torch.from_numpy(np.array(a)).cuda()   # noqa: E731
    pool = dsa.PagePool.of(put(stack), put(np.array([count], np.int32)))
    seq, t = put(lens), put(table)
    kw = dict(seq_lens_out=seq, free_count_out=pool.count) if in_place else {}
    got = dsa.step_plan(pool, seq, put(new), t, P, rows, check=check, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(pool.pages.cpu().numpy(), stack)
    if not in_place:
        assert np.array_equal(seq.cpu().numpy(), lens) and int(pool.count.item()) == count
    return [x.cpu().numpy() for x in (got.seq_lens, got.query_start_loc, got.slot_mapping, got.positions)] + \
        [int(got.free_count.item()), t.cpu().numpy()]


def same(got, want):
    for name, g, w in zip(("seq_lens", "starts", "slots", "positions", "count", "table"), got, want):
        assert np.array_equal(g, w), name


@pytest.mark.parametrize("B,P,hi,news,extra", [(1, 16, 0, [1], 0), (1, 1, 3, [5], 2), (8, 64, 8192, [1], 0), (33, 16, 300, [1, 4, 0, 37], 9),
                                               (256, 64, 5000, [1, 1, 0, 4, 197], 100), (1500, 32, 200, [2, 0, 7], 0),
                                               (4096, 16, 400, [17, 0, 3], 11), (5, 1024, 5000, [2100, 0], 3), (2, 128, 1000, [30000], 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_matches_the_oracle(B, P, hi, news, extra, in_place):
    lens, new, table, stack, count, _ = make(B, B, P, hi, news)
    rows = int(new.sum()) + extra
    want = d.step_plan(lens, new, P, table, stack, count, rows)
    assert not want[-1]
    same(plan(lens, new, table, stack, count, P, rows, check=True, in_place=in_place), want)


@pytest.mark.parametrize("B", [7, 300, 2500])
@pytest.mark.parametrize("short", ["pages", "rows"])
def test_the_longest_prefix_is_admitted(B, short):
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    lens, new, table, stack, count, _ = make(B + 1, B, 16, 60, [9, 0, 30, 1])
    rows = int(new.sum())
    if short == "pages":
        count = int((-(-(lens + new) // 16) - -(-lens // 16)).sum()) // 2
    else:
        rows //= 2
    want = d.step_plan(lens, new, 16, table, stack, count, rows)
    assert want[-1] and want[1][-1] > 0
    same(plan(lens, new, table, stack, count, 16, rows), want)
    with pytest.raises(dsa.DsaError, match="POOL_EMPTY" if short == "pages" else "ROWS_FULL"):
        plan(lens, new, table, stack, count, 16, rows, check=True)
    torch.cuda.synchronize()


def test_requests_whose_lengths_make_no_sense_rest():
    import deepseek_sparse_mla_gb300 as dsa
    lens, new, table, stack, count, _ = make(5, 12, 16, 60, [3])
    new[2], lens[5], new[7] = -1, -4, 10 ** 6
    rows = 64
    want = list(d.step_plan(lens, new, 16, table, stack, count, rows))
    same(plan(lens, new, table, stack, count, 16, rows), want)
    with pytest.raises(dsa.DsaError, match="BAD_LENGTH"):
        plan(lens, new, table, stack, count, 16, rows, check=True)


@pytest.mark.parametrize("B,P", [(1, 16), (40, 16), (700, 64)])
def test_released_pages_come_back(B, P):
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    lens, new, table, stack, count, total = make(B + 9, B, P, 900, [0])
    rng = np.random.default_rng(B)
    done = (rng.random(B) < 0.5).astype(np.int32)
    done[0] = 1
    put = lambda a: torch.from_numpy(np.array(a)).cuda()   # noqa: E731
    stack = np.concatenate([stack[:count], np.full(total - count, -9, np.int32)])
    pool, seq, t = dsa.PagePool.of(put(stack), put(np.array([count], np.int32))), put(lens), put(table)
    dsa.pages_release(pool, put(done), seq, t, P, total, check=True)
    back = [int(p) for b in range(B) if done[b] for p in table[b, :-(-int(lens[b]) // P)]]
    assert int(pool.count.item()) == count + len(back)
    assert list(pool.pages.cpu().numpy()[:count + len(back)]) == list(stack[:count]) + back
    want = table.copy()
    for b in range(B):
        if done[b]:
            want[b, :-(-int(lens[b]) // P)] = -1
    assert np.array_equal(t.cpu().numpy(), want)
    assert np.array_equal(seq.cpu().numpy(), np.where(done, 0, lens))


def test_release_keeps_what_the_stack_has_no_room_for_and_drops_bad_ids():
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    put = lambda a: torch.from_numpy(np.array(a, np.int32)).cuda()   # noqa: E731
    table = put([[3, 99, 4], [5, 6, 7], [1, -1, -1]])
    seq = put([33, 40, 5])
    pool = dsa.PagePool.of(put([8, 0, 0, 0]), put([1]))
    with pytest.raises(dsa.DsaError, match="BAD_PAGE.*POOL_FULL"):
        dsa.pages_release(pool, put([1, 1, 1]), seq, table, 16, 10, check=True)
    torch.cuda.synchronize()
    assert pool.pages.tolist() == [8, 3, 4, 0] and pool.count.tolist() == [3]
    assert seq.tolist() == [0, 40, 5] and table.tolist() == [[-1, -1, -1], [5, 6, 7], [1, -1, -1]]
