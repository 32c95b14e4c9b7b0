"""Error bounds of requests of many rows over the 4-bit cache, which hold more than the few-row kernel's (dense_cases.bounds)."""
import numpy as np

from oracle import kv4_oracle as f


def score_errors(case, Z, scale):
    """Of scores (no cap or bias): fp32 sums of exact products, 2^-15 of sum |q k|, exp2's 2^-20, and q's own: its smaller e4m3 term has
    steps of 2^-9 where the row's largest value is 2^7 or more, so half a step is at most 2^-17 of that value, times sum |k|."""
    q_max = np.abs(case.q).max(-1)
    dz = 2.0 ** -15 * Z + 2.0 ** -20
    for b, L in enumerate(int(v) for v in case.seq_lens):
        s = np.arange(L)
        pages = case.table[b, s // case.P]
        rows = slice(case.starts[b], case.starts[b + 1])
        for h in range(case.kv):
            k = f.values(case.cache["k"][pages, h, s % case.P]) * np.repeat(np.exp2(case.cache["ks"][pages, h, s % case.P].astype(np.float64) - 127), 32, -1)
            heads = slice(h * case.group, (h + 1) * case.group)
            dz[rows, heads] += scale * 2.0 ** -17 * q_max[rows, heads] * np.abs(k).sum(-1).max()
    return dz


def prompt_errors(case, got, want, scale, v_error=0.0):
    """|got - want| over its bound:
    p       fp16 of 2^8 p: half a step, 2^-11 of it, and below fp16's normal numbers 2^-33 of the largest p (2^-32 of C is taken)
    v       exact where its scale is 2^-26 of the largest or more; else v_error
    sums    fp32 over at most 2^11 keys, of p in chains of a quarter of them: 2^-13 with exp2's error
    output  bf16, half a step: 2^-8 of the value."""
    out, _, A, C, Z = want
    dz = score_errors(case, Z, scale)[..., None]
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2.0 ** -13 + 2 * dz) * A + 2.0 ** -32 * C + v_error * (1 + 2.0 ** -8)
    return np.abs(got - out) / np.maximum(tol, 1e-300)
