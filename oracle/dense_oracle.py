"""Float64 CPU oracle of the step planner, the block-scaled 8-bit K/V cache and the dense attention over it.
TEST INFRASTRUCTURE ONLY: it shares no code with the CUDA path, and every step is the plain definition.

* step plan -- requests are taken in order while their new rows fit ``num_rows`` and their new pages the stack; new
  pages come off the top of the stack, in request order ("GLM-5.2 on vLLM Ascend: Request-to-Backend Inference Path",
  section 4 "NPU batch preparation and attention metadata": cumulative query lengths, sequence lengths, block tables
  and per-token slot mappings).
* append -- per page and head: ``want = 2^ceil(log2(amax / 448))`` of the new tokens' finite values, at least 2^-126;
  a page that holds older tokens keeps the larger of its scale and ``want``, and its older codes are re-coded when the
  scale grew.
* attention -- ``z = scale * q . (k_code * k_scale)``, then ``cap * tanh(z / cap)``, then ``- slope * |pos - s|``;
  softmax over the visible positions of ``v_code * v_scale``; a row that sees nothing is 0 with an lse of -inf
  ("GLM-5.2 on vLLM Ascend", the draft layers' dense paged attention with grouped heads).
"""
from __future__ import annotations

import numpy as np

from . import dsa_oracle as o

MIN_SCALE = 2.0 ** -126


def step_plan(seq_lens, new_lens, page_size, table, free, count, num_rows):
    """(seq_lens, query_start_loc, slots, positions, count, table, refused) after the step; table is copied."""
    table = np.array(table)
    lens, starts = [int(L) for L in seq_lens], [0]
    slots, positions = np.full(num_rows, -1, np.int64), np.full(num_rows, -1, np.int32)
    full, refused = False, []
    for b, (L, n) in enumerate(zip(seq_lens, new_lens)):
        L, n = int(L), int(n)
        have, want = -(-L // page_size), -(-(L + n) // page_size)
        if L < 0 or n < 0 or (n > 0 and want > table.shape[1]):
            refused.append(b)
            n, want = 0, have
        if starts[-1] + n > num_rows or want - have > count:
            full = True
        if full and n:
            refused.append(b)
            n = 0
        if n:
            for lp in range(have, want):
                count -= 1
                table[b, lp] = free[count]
            for i in range(n):
                positions[starts[-1] + i] = L + i
                slots[starts[-1] + i] = int(table[b, (L + i) // page_size]) * page_size + (L + i) % page_size
        lens[b] = L + n
        starts.append(starts[-1] + n)
    return np.array(lens, np.int32), np.array(starts, np.int32), slots, positions, count, table, refused


def block_scale(x) -> float:
    """The power of two that a block's values ask for."""
    x = np.abs(np.asarray(x, np.float64))
    x = x[np.isfinite(x)]
    top = float(x.max()) if x.size else 0.0
    if top == 0.0:
        return MIN_SCALE
    k = -126
    while 448.0 * 2.0 ** k < top:
        k += 1
    return 2.0 ** k


def encode(x) -> np.ndarray:
    """e4m3 codes of values already divided by their scale: nearest-even, saturating, infinities too; NaN is 0x7F."""
    x = np.asarray(x, np.float32)
    nan = np.isnan(x)
    x = np.where(np.isinf(x), np.copysign(np.float32(448.0), x), np.where(nan, np.float32(0.0), x))
    return np.where(nan, np.uint8(0x7F), o.f32_to_e4m3(x)).astype(np.uint8)


def append(codes, scales, table, seq_lens, starts, x):
    """codes [pages, heads, P, 128] uint8 and scales [pages, heads] float32 after appending x [rows, heads, 128] float64;
    both are copied."""
    codes, scales = np.array(codes), np.array(scales)
    pages, heads, P, _ = codes.shape
    for b, L in enumerate(int(v) for v in seq_lens):
        n = int(starts[b + 1] - starts[b])
        at, r = L - n, int(starts[b])
        if at < 0:
            continue
        while at < L:
            lp, off = at // P, at % P
            m = min(P - off, L - at)
            page = int(table[b, lp]) if lp < table.shape[1] else -1
            if 0 <= page < pages:
                for h in range(heads):
                    new = x[r:r + m, h]
                    want, have = block_scale(new), float(scales[page, h])
                    s = max(want, have) if off else want
                    if off and have < s:
                        ratio = np.float32(np.float32(have) / np.float32(s))
                        old = o.e4m3_to_f64(codes[page, h, :off]).astype(np.float32)
                        codes[page, h, :off] = encode(old * ratio)
                    codes[page, h, off:off + m] = encode(new.astype(np.float32) / np.float32(s))
                    scales[page, h] = s
            at, r = at + m, r + m
    return codes, scales


def attention(k_codes, v_codes, k_scales, v_scales, table, seq_lens, starts, q, scale, softcap=0.0, slopes=None, prefix=None):
    """out [rows, q_heads, 128], lse [rows, q_heads], and for the error bounds: A = sum_s p_s |v_s| like out, C (the
    largest p_s times the largest v scale, times sum_s |v_code_s|) like out, and Z like lse, the largest sum_d |q_d k_sd| *
    scale of a key that counts.  Rows behind the last request's are NaN."""
    pages, heads, P, D = k_codes.shape
    q = np.asarray(q, np.float64)
    rows, q_heads = q.shape[:2]
    g = q_heads // heads
    out, A, C = (np.full((rows, q_heads, D), np.nan) for _ in range(3))
    lse, Z = (np.full((rows, q_heads), np.nan) for _ in range(2))
    for b, L in enumerate(int(v) for v in seq_lens):
        n = int(starts[b + 1] - starts[b])
        ids = np.array([table[b, s // P] if s // P < table.shape[1] else -1 for s in range(L)], np.int64)
        there = (ids >= 0) & (ids < pages)
        off = np.arange(L) % P
        safe = np.where(there, ids, 0)
        for h in range(heads):
            kc, vc = o.e4m3_to_f64(k_codes[safe, h, off]), o.e4m3_to_f64(v_codes[safe, h, off])
            k, vs = kc * k_scales[safe, h].astype(np.float64)[:, None], v_scales[safe, h].astype(np.float64)[:, None]
            for i in range(n):
                pos = L - n + i
                end = pos if prefix is None else max(pos, min(int(prefix[b]), L) - 1)
                see = there & (np.arange(L) <= end)
                r = int(starts[b]) + i
                for head in range(h * g, (h + 1) * g):
                    if not see.any():
                        out[r, head], lse[r, head], A[r, head], C[r, head], Z[r, head] = 0.0, -np.inf, 0.0, 0.0, 0.0
                        continue
                    with np.errstate(invalid="ignore", over="ignore"):
                        z = scale * (k[see] @ q[r, head])
                        if softcap:
                            z = softcap * np.tanh(z / softcap)
                        if slopes is not None:
                            z = z - float(slopes[head]) * np.abs(pos - np.arange(L)[see])
                        m = z.max()
                        p = np.exp(z - m)
                        total = p.sum()
                        p = p / total
                        out[r, head] = p @ (vc[see] * vs[see])
                        lse[r, head] = m + np.log(total)
                        A[r, head] = p @ np.abs(vc[see] * vs[see])
                        C[r, head] = p.max() * np.abs(vs[see]).max() * np.abs(vc[see]).sum(0)
                        Z[r, head] = scale * (np.abs(k[see][p > 1e-9]) @ np.abs(q[r, head])).max(initial=0.0)
    return out, lse, A, C, Z
