"""The step planner, the 8-bit append and the dense attention together, as a serving loop runs them: prompts in pieces, then
decode steps, with requests that end and return their pages; eagerly and as a captured graph."""
import numpy as np
import pytest

import workloads as wlm
from dense_cases import check_attention
from oracle import dense_oracle as d
from oracle import dsa_oracle as o

pytestmark = pytest.mark.gpu


class Loop:
    """The loop's state on the device and, step for step, in the oracle."""

    def __init__(self, B, P, kv, group, pages, width, rows, longest, seed):
        import torch
        import deepseek_sparse_mla_gb300 as dsa
        self.B, self.P, self.kv, self.group, self.rows, self.longest = B, P, kv, group, rows, longest
        self.heads, self.pages = kv * group, pages
        self.rng = np.random.default_rng(seed)
        self.pool = dsa.PagePool(pages)
        self.cache = dsa.BlockKvCache(pages, P, kv)
        self.cache.k_codes.fill_(0x7F), self.cache.v_codes.fill_(0x7F)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.seq, self.new = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.table, self.done = torch.full((B, width), -1, **i32), torch.zeros(B, **i32)
        self.starts, self.positions = torch.zeros(B + 1, **i32), torch.zeros(rows, **i32)
        self.slots = torch.zeros(rows, dtype=torch.int64, device="cuda")
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.qkv = torch.zeros(rows, self.heads + 2 * kv, 128, **bf)
        self.out, self.lse = torch.zeros(rows, self.heads, 128, **bf), torch.zeros(rows, self.heads, device="cuda")
        self.ws = torch.empty(dsa.paged_attention_workspace_bytes(self.heads, kv, longest), dtype=torch.uint8, device="cuda")
        self.max_len = width * P
        self.h_seq, self.h_table, self.h_count = np.zeros(B, np.int64), np.full((B, width), -1, np.int32), pages
        self.h_free = np.arange(pages - 1, -1, -1).astype(np.int32)
        self.h_codes = {n: np.full((pages, kv, P, 128), 0x7F, np.uint8) for n in "kv"}
        self.h_scales = {n: np.ones((pages, kv), np.float32) for n in "kv"}

    def step(self):
        """One step on the device, all of it on the current stream."""
        import deepseek_sparse_mla_gb300 as dsa
        h, kv = self.heads, self.kv
        dsa.step_plan(self.pool, self.seq, self.new, self.table, self.P, self.rows, seq_lens_out=self.seq, query_start_loc=self.starts,
                      slot_mapping=self.slots, positions=self.positions, free_count_out=self.pool.count)
        batch = dsa.Batch(self.table, self.seq, self.starts, num_rows=self.rows, max_seq_len=self.max_len)
        dsa.kv8_append(self.cache, batch, self.qkv[:, h:h + kv], self.qkv[:, h + kv:])
        dsa.paged_attention(self.cache, batch, self.qkv[:, :h], max_query_len=self.longest, out=self.out, lse=self.lse, workspace=self.ws)

    def feed(self, new):
        self.h_new = np.array(new, np.int64)
        self.new.copy_(wlm_put(self.h_new.astype(np.int32)))
        self.bits = wlm.bf16_bits(self.rng.standard_normal((self.rows, self.heads + 2 * self.kv, 128)).astype(np.float32))
        self.qkv.copy_(wlm.bits_to_torch(self.bits, "cuda"))

    def check(self):
        """The oracle's step, then everything that the device holds against it."""
        import torch
        torch.cuda.synchronize()
        lens, starts, slots, positions, count, table, refused = d.step_plan(self.h_seq, self.h_new, self.P, self.h_table,
                                                                            self.h_free[:self.h_count], self.h_count, self.rows)
        assert np.array_equal(self.seq.cpu().numpy(), lens) and np.array_equal(self.starts.cpu().numpy(), starts)
        assert np.array_equal(self.slots.cpu().numpy(), slots) and np.array_equal(self.positions.cpu().numpy(), positions)
        assert np.array_equal(self.table.cpu().numpy(), table) and int(self.pool.count.item()) == count
        self.h_seq, self.h_table, self.h_count = np.array(lens, np.int64), table, count
        x, h, kv = o.bf16_to_f64(self.bits), self.heads, self.kv
        for n, part, codes, scales in (("k", x[:, h:h + kv], self.cache.k_codes, self.cache.k_scales),
                                       ("v", x[:, h + kv:], self.cache.v_codes, self.cache.v_scales)):
            self.h_codes[n], self.h_scales[n] = d.append(self.h_codes[n], self.h_scales[n], table, lens, starts, part)
            assert np.array_equal(codes.cpu().numpy(), self.h_codes[n]) and np.array_equal(scales.cpu().numpy(), self.h_scales[n])
        want = d.attention(self.h_codes["k"], self.h_codes["v"], self.h_scales["k"], self.h_scales["v"], table, lens, starts,
                           x[:, :h], 128 ** -0.5)
        check_attention(o.bf16_to_f64(wlm.torch_to_bits(self.out)), self.lse.cpu().numpy().astype(np.float64), want)
        return refused

    def release(self, done):
        import torch
        import deepseek_sparse_mla_gb300 as dsa
        self.done.copy_(wlm_put(np.array(done, np.int32)))
        dsa.pages_release(self.pool, self.done, self.seq, self.table, self.P, self.pages, check=True)
        torch.cuda.synchronize()
        back = [p for b in range(self.B) if done[b] for p in self.h_table[b, :-(-int(self.h_seq[b]) // self.P)]]
        self.h_free = self.h_free.copy()
        self.h_free[self.h_count:self.h_count + len(back)] = back
        self.h_count += len(back)
        for b in range(self.B):
            if done[b]:
                self.h_table[b, :-(-int(self.h_seq[b]) // self.P)] = -1
                self.h_seq[b] = 0
        assert int(self.pool.count.item()) == self.h_count and np.array_equal(self.table.cpu().numpy(), self.h_table)
        assert list(self.pool.pages[:self.h_count].cpu().numpy()) == list(self.h_free[:self.h_count])


def wlm_put(a):
    import torch
    return torch.from_numpy(np.array(a)).cuda()


def test_prompts_in_pieces_then_decode_with_requests_that_end():
    loop = Loop(B=4, P=16, kv=2, group=8, pages=40, width=20, rows=64, longest=40, seed=1)
    for new in ([30, 0, 0, 5], [33, 1, 12, 1], [1, 40, 1, 3], [1, 1, 1, 1], [1, 4, 0, 1]):
        loop.feed(new)
        loop.step()
        loop.check()
    loop.release([1, 0, 0, 1])
    for new in ([17, 1, 1, 0], [1, 2, 3, 39], [1, 1, 1, 1]):
        loop.feed(new)
        loop.step()
        loop.check()
    loop.release([1, 1, 1, 1])
    assert loop.h_count == 40


def test_requests_wait_where_the_pool_is_empty_and_go_on_when_pages_come_back():
    loop = Loop(B=3, P=16, kv=1, group=4, pages=6, width=6, rows=80, longest=40, seed=2)
    loop.feed([40, 33, 16])
    loop.step()
    loop.check()
    assert loop.h_seq.tolist() == [40, 33, 0]                # the third found no page
    loop.release([1, 0, 0])
    loop.feed([0, 1, 16])
    loop.step()
    loop.check()
    assert loop.h_seq.tolist() == [0, 34, 16]


@pytest.mark.parametrize("longest", [2, 20])
def test_a_captured_step_replayed(longest):
    import torch
    loop = Loop(B=5, P=32, kv=1, group=8, pages=60, width=12, rows=40, longest=longest, seed=3)
    loop.feed([0] * 5)
    g = torch.cuda.CUDAGraph()
    loop.step()                                              # a step without tokens changes nothing
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        loop.step()
    rng = np.random.default_rng(3)
    for _ in range(8):
        loop.feed(rng.integers(0, min(longest, 8) + 1, 5))
        g.replay()
        loop.check()
