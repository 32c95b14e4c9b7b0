"""Shared by the tests of the 4-bit K/V cache: seeded batches over a pool that earlier appends filled."""
import numpy as np

import workloads as wlm
from oracle import dsa_oracle as o
from oracle import kv4_oracle as f


class Kv4Case:
    """Requests of seq_lens tokens, the last q_lens of them this step's rows, over a pool of shuffled pages filled as earlier
    appends leave it (each token at a magnitude of its own, a few wide dims of K); slots behind a request hold NaN scales."""

    def __init__(self, seed, seq_lens, q_lens, P, kv, group, spare=3, extra_rows=0, spread=0.7, extra_width=2):
        rng = self.rng = np.random.default_rng(seed)
        self.P, self.kv, self.group, self.heads = P, kv, group, kv * group
        self.seq_lens, self.q_lens = np.array(seq_lens, np.int32), np.array(q_lens, np.int32)
        self.starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.rows = int(self.starts[-1]) + extra_rows
        held = [-(-int(L) // P) for L in seq_lens]
        self.pages = sum(held) + spare
        perm = rng.permutation(self.pages)
        self.table = np.full((len(held), max(max(held), 1) + extra_width), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = perm[at:at + n]
            at += n
        shape = (self.pages, kv, P)
        self.cache = {"k": rng.integers(0, 256, (*shape, 64)).astype(np.uint8), "v": rng.integers(0, 256, (*shape, 64)).astype(np.uint8),
                      "ks": np.full((*shape, 4), f.NAN_SCALE, np.uint8), "vs": np.full(shape, np.nan)}
        wide = np.where(rng.random((kv, 128)) < 1 / 16, 4.0, 0.8)
        for b, L in enumerate(int(v) for v in seq_lens):
            s = np.arange(L)
            ids = self.table[b, s // P]
            for h in range(kv):
                k = rng.standard_normal((L, 128)) * wide[h]
                v = rng.standard_normal((L, 128)) * 2.0 ** (spread * rng.standard_normal((L, 1)))
                # the quantisers of the oracle, a head's tokens at once
                e = np.clip(np.ceil(np.log2(np.abs(k.reshape(L, 4, 32)).max(-1) / 6.0)), f.LOW, f.HIGH)
                self.cache["k"][ids, h, s % P] = f.two_a_byte(f.encode(k / np.repeat(2.0 ** e, 32, -1)))
                self.cache["ks"][ids, h, s % P] = (e + 127).astype(np.uint8)
                vs = np.array([f._bf16(x) for x in np.abs(v).max(-1) / 6.0])
                self.cache["v"][ids, h, s % P] = f.two_a_byte(f.encode(v / vs[:, None])) if L else 0
                self.cache["vs"][ids, h, s % P] = vs
        self.q_bits = wlm.bf16_bits(rng.standard_normal((self.rows, self.heads, 128)).astype(np.float32))
        self.new = {n: wlm.bf16_bits(rng.standard_normal((self.rows, kv, 128)).astype(np.float32)) for n in "kv"}
        self.slopes = (2.0 ** (-8.0 * (np.arange(self.heads) + 1) / self.heads)).astype(np.float32)

    @property
    def q(self):
        return o.bf16_to_f64(self.q_bits)

    def oracle(self, scale=128 ** -0.5, **mods):
        return f.attention(self.cache, self.table, self.seq_lens, self.starts, self.q, scale, **mods)

    def gpu(self, max_seq_len=None):
        """(cache, batch, q) on the device."""
        import torch
        import deepseek_sparse_mla_gb300 as dsa
        put = lambda a: torch.from_numpy(np.array(a)).cuda()   # noqa: E731
        vs = put(self.cache["vs"].astype(np.float32)).to(torch.bfloat16)
        cache = dsa.Kv4Cache.of(put(self.cache["k"]), put(self.cache["v"]), put(self.cache["ks"]), vs)
        batch = dsa.Batch(put(self.table), put(self.seq_lens), put(self.starts), num_rows=self.rows,
                          max_seq_len=max_seq_len or max(1, int(self.seq_lens.max())))
        return cache, batch, wlm.bits_to_torch(self.q_bits, "cuda")


def rope_table(positions, dim, seed=None):
    """float32 [positions, dim]: cos, then sin."""
    turn = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
    return np.concatenate([np.cos(turn), np.sin(turn)], 1).astype(np.float32)
