"""Shared by the tests of the dense layer: seeded batches over a paged 8-bit K/V cache, and the error bounds."""
import numpy as np

import workloads as wlm
from oracle import dense_oracle as d
from oracle import dsa_oracle as o


class DenseCase:
    """Requests of seq_lens tokens, the last q_lens of them this step's rows, over a pool of shuffled pages filled as
    earlier appends leave it (each page at a magnitude of its own); slots behind a request hold NaN codes."""

    def __init__(self, seed, seq_lens, q_lens, P, kv, group, spare=3, extra_rows=0, spread=1.0, extra_width=2):
        rng = np.random.default_rng(seed)
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
        shape = (self.pages, kv, P, 128)
        self.codes, self.scales = {}, {}
        for name in "kv":
            self.codes[name] = np.full(shape, 0x7F, np.uint8)
            self.scales[name] = np.ones(shape[:2], np.float32)
            for b, L in enumerate(int(v) for v in seq_lens):
                for lp in range(held[b]):
                    n, page = min(P, L - lp * P), self.table[b, lp]
                    x = rng.standard_normal((kv, n, 128)) * 2.0 ** (spread * rng.standard_normal((kv, 1, 1)))
                    for h in range(kv):
                        s = d.block_scale(x[h])
                        self.codes[name][page, h, :n] = d.encode(x[h] / s)
                        self.scales[name][page, h] = s
        self.q_bits = wlm.bf16_bits(rng.standard_normal((self.rows, self.heads, 128)).astype(np.float32))
        self.new = {n: wlm.bf16_bits(rng.standard_normal((self.rows, kv, 128)).astype(np.float32)) for n in "kv"}
        self.slopes = (2.0 ** (-8.0 * (np.arange(self.heads) + 1) / self.heads)).astype(np.float32)

    @property
    def q(self):
        return o.bf16_to_f64(self.q_bits)

    def oracle(self, scale=128 ** -0.5, **mods):
        return d.attention(self.codes["k"], self.codes["v"], self.scales["k"], self.scales["v"], self.table, self.seq_lens,
                           self.starts, self.q, scale, **mods)

    def gpu(self, max_seq_len=None):
        """(cache, batch, q) on the device."""
        import torch
        import deepseek_sparse_mla_gb300 as dsa
        put = lambda a: torch.from_numpy(np.array(a)).cuda()   # noqa: E731
        cache = dsa.BlockKvCache.of(put(self.codes["k"]), put(self.codes["v"]), put(self.scales["k"]), put(self.scales["v"]))
        batch = dsa.Batch(put(self.table), put(self.seq_lens), put(self.starts), num_rows=self.rows,
                          max_seq_len=max(1, int(self.seq_lens.max())))
        return cache, batch, wlm.bits_to_torch(self.q_bits, "cuda")


def bounds(out, lse, A, C, Z, softcap=0.0, reach=0.0):
    """Error bounds of (out, lse), from the formulas:
    scores   fp32 sums of 128 exact products (and q's own 2^-22 of its row's largest): 2^-15 of sum |q k|, plus the
             approximations of exp2 and of the cap (2^-20 of it), plus the bias' rounding (2^-22 of the largest)
    values   a contribution keeps two e4m3 terms: half a step of 4 bits twice, 2^-4 * 2^-4 = 2^-8 of it, and an absolute
             half step of 2^-20 of the reference, which is within 2^2 of the largest contribution: 2^-18
    output   bf16, half a step: 2^-8 of the value (2^-9 above the step's base)."""
    dz = 2.0 ** -15 * Z + 2.0 ** -20 * (1.0 + softcap) + 2.0 ** -22 * reach
    tol_lse = dz + 2.0 ** -20 * (1.0 + np.where(np.isfinite(lse), np.abs(lse), 0.0))
    tol_out = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 * 1.02 + 2 * dz[..., None]) * A + 2.0 ** -18 * C + 1e-30
    return tol_out, tol_lse


def check_attention(got, got_lse, want, softcap=0.0, reach=0.0):
    out, lse, A, C, Z = want
    live = ~np.isnan(Z)
    tol_out, tol_lse = bounds(out, lse, A, C, Z, softcap, reach)
    err = np.abs(got[live] - out[live])
    assert np.all(np.isfinite(got[live])), "not finite"
    over = err / tol_out[live]
    assert over.max(initial=0.0) <= 1.0, f"outputs off by {over.max():.3f} of the bound ({err.max():.3e})"
    if got_lse is not None:
        empty = np.isneginf(lse) & live
        assert np.all(np.isneginf(got_lse[empty])) and np.all(got[empty] == 0.0)
        full = live & ~empty
        over = np.abs(got_lse[full] - lse[full]) / tol_lse[full]
        assert over.max(initial=0.0) <= 1.0, f"lse off by {over.max():.3f} of the bound"
    return float((err / np.maximum(tol_out[live], 1e-300)).max(initial=0.0))
