"""The step planner, the rotating appends and the dense attention over both caches together, as a serving loop runs them:
prompts in pieces, then decode steps, eagerly and as a captured graph."""
import numpy as np
import pytest

import workloads as wlm
from dense_cases import check_attention
from kv4_cases import rope_table
from oracle import dense_oracle as d
from oracle import dsa_oracle as o
from oracle import kv4_oracle as f

pytestmark = pytest.mark.gpu


def put(a):
    import torch
    return torch.from_numpy(np.array(a)).cuda()


class Loop:
    """The loop's state on the device and, step for step, in the oracle."""

    def __init__(self, bits, B, P, kv, group, pages, width, rows, longest, dim, interleaved, seed):
        import torch
        import deepseek_sparse_mla_gb300 as dsa
        self.bits, self.B, self.P, self.kv, self.rows, self.longest, self.heads = bits, B, P, kv, rows, longest, kv * group
        self.rng, self.interleaved = np.random.default_rng(seed), interleaved
        self.pool, self.max_len = dsa.PagePool(pages), width * P
        self.cache = (dsa.Kv4Cache if bits == 4 else dsa.BlockKvCache)(pages, P, kv)
        self.table_cs = rope_table(self.max_len, dim)
        self.rope = dsa.RotaryTable.of(put(self.table_cs), interleaved)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.seq, self.new, self.table = torch.zeros(B, **i32), torch.zeros(B, **i32), torch.full((B, width), -1, **i32)
        self.starts, self.positions = torch.zeros(B + 1, **i32), torch.zeros(rows, **i32)
        self.slots = torch.zeros(rows, dtype=torch.int64, device="cuda")
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.qkv = torch.zeros(rows, self.heads + 2 * kv, 128, **bf)
        self.out, self.lse = torch.zeros(rows, self.heads, 128, **bf), torch.zeros(rows, self.heads, device="cuda")
        self.ws = torch.empty(dsa.paged_attention_workspace_bytes(self.heads, kv, longest), dtype=torch.uint8, device="cuda")
        self.h_seq, self.h_table, self.h_count = np.zeros(B, np.int64), np.full((B, width), -1, np.int32), pages
        self.h_free = np.arange(pages - 1, -1, -1).astype(np.int32)
        shape = (pages, kv, P)
        self.h4 = {"k": np.zeros((*shape, 64), np.uint8), "v": np.zeros((*shape, 64), np.uint8), "ks": np.full((*shape, 4), 127, np.uint8), "vs": np.ones(shape)}
        self.h8 = {n: (np.zeros((*shape, 128), np.uint8), np.ones((pages, kv), np.float32)) for n in "kv"}

    def step(self):
        """One step on the device, all of it on the current stream; the queries are rotated in place."""
        import deepseek_sparse_mla_gb300 as dsa
        h, kv = self.heads, self.kv
        dsa.step_plan(self.pool, self.seq, self.new, self.table, self.P, self.rows, seq_lens_out=self.seq, query_start_loc=self.starts,
                      slot_mapping=self.slots, positions=self.positions, free_count_out=self.pool.count)
        batch = dsa.Batch(self.table, self.seq, self.starts, num_rows=self.rows, max_seq_len=self.max_len)
        append = dsa.kv4_append if self.bits == 4 else dsa.kv8_append
        q = append(self.cache, batch, self.qkv[:, h:h + kv], self.qkv[:, h + kv:], rope=self.rope, q=self.qkv[:, :h], q_out=self.qkv[:, :h])
        dsa.paged_attention(self.cache, batch, q, max_query_len=self.longest, out=self.out, lse=self.lse, workspace=self.ws)

    def feed(self, new):
        self.h_new = np.array(new, np.int64)
        self.new.copy_(put(self.h_new.astype(np.int32)))
        self.in_bits = wlm.bf16_bits(self.rng.standard_normal((self.rows, self.heads + 2 * self.kv, 128)).astype(np.float32))
        self.qkv.copy_(wlm.bits_to_torch(self.in_bits, "cuda"))

    def check(self):
        """The oracle's step, then everything that the device holds against it."""
        import torch
        torch.cuda.synchronize()
        lens, starts, slots, positions, count, table, _ = d.step_plan(self.h_seq, self.h_new, self.P, self.h_table,
                                                                      self.h_free[:self.h_count], self.h_count, self.rows)
        assert np.array_equal(self.seq.cpu().numpy(), lens) and np.array_equal(self.positions.cpu().numpy(), positions)
        self.h_seq, self.h_table, self.h_count = np.array(lens, np.int64), table, count
        x, h, kv, live = o.bf16_to_f64(self.in_bits), self.heads, self.kv, positions >= 0
        turned = f.rotate32(x, self.table_cs, np.maximum(positions, 0), self.interleaved)
        q = o.bf16_to_f64(wlm.bf16_bits(turned[:, :h]))
        got_q = o.bf16_to_f64(wlm.torch_to_bits(self.qkv[:, :h].contiguous()))
        assert np.array_equal(got_q[live], q[live]) and np.array_equal(got_q[~live], x[~live, :h])
        k, v, c = turned[:, h:h + kv].astype(np.float64), x[:, h + kv:], self.cache
        if self.bits == 4:
            self.h4 = f.append(self.h4, table, lens, starts, k, v)
            for name, t in (("k", c.k_codes), ("v", c.v_codes), ("ks", c.k_scales), ("vs", c.v_scales.double())):
                assert np.array_equal(t.cpu().numpy(), self.h4[name]), name
            want = f.attention(self.h4, table, lens, starts, q, 128 ** -0.5)
        else:
            for name, part, codes, scales in (("k", k, c.k_codes, c.k_scales), ("v", v, c.v_codes, c.v_scales)):
                self.h8[name] = d.append(*self.h8[name], table, lens, starts, part)
                assert np.array_equal(codes.cpu().numpy(), self.h8[name][0]) and np.array_equal(scales.cpu().numpy(), self.h8[name][1])
            want = d.attention(self.h8["k"][0], self.h8["v"][0], self.h8["k"][1], self.h8["v"][1], table, lens, starts, q, 128 ** -0.5)
        check_attention(o.bf16_to_f64(wlm.torch_to_bits(self.out)), self.lse.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim,interleaved", [(128, False), (64, True)])
def test_prompts_in_pieces_then_decode(bits, dim, interleaved):
    loop = Loop(bits, B=4, P=16, kv=2, group=8, pages=40, width=20, rows=64, longest=40, dim=dim, interleaved=interleaved, seed=1)
    for new in ([30, 0, 0, 5], [33, 1, 12, 1], [1, 40, 1, 3], [1, 1, 1, 1], [1, 4, 0, 1]):
        loop.feed(new)
        loop.step()
        loop.check()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("longest", [2, 20])
def test_a_captured_step_replayed(bits, longest):
    import torch
    loop = Loop(bits, B=5, P=32, kv=1, group=8, pages=60, width=12, rows=40, longest=longest, dim=96, interleaved=False, seed=3)
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

