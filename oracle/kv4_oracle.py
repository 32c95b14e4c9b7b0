"""Float64 CPU oracle of the position rotation, the paged 4-bit K/V cache and the dense attention over it.
TEST INFRASTRUCTURE ONLY: it shares no code with the CUDA path, and every step is the plain definition.

* rotation -- ``(a, b) -> (a c - b s, b c + a s)`` of dims (i, i + dim/2) or (2i, 2i + 1); ``rotate32`` takes each product and
  each sum in float32, which the quantised keys follow, and ``rotate`` the definition ("vLLM Inference Path: GLM-5.2
  as an Example", "MLA Projections and KV State": RoPE on part of a head).
* append -- K: per 32 dims ``2^ceil(log2(amax / 6))``, exponent held in [-15, 13]; V: per token and head ``bf16(amax / 6)``, at
  least 2^-126; codes are the nearest e2m1 value of ``x / scale``, ties to the even code, saturating.
* attention -- as in ``dense_oracle``, over ``k_code * 2^e`` and ``v_code * v_scale``.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])
LOW, HIGH, NAN_SCALE = -15, 13, 255


def _pairs(x, dim, interleaved):
    return (x[..., 0:dim:2], x[..., 1:dim:2]) if interleaved else (x[..., :dim // 2], x[..., dim // 2:dim])


def _turn(x, table, pos, interleaved, dtype):
    x = np.array(x, dtype)
    dim = table.shape[1]
    angles = table[pos].astype(dtype)[:, None]
    c, s = angles[..., :dim // 2], angles[..., dim // 2:]
    a, b = (np.array(v) for v in _pairs(x, dim, interleaved))
    ra, rb = _pairs(x, dim, interleaved)
    with np.errstate(invalid="ignore", over="ignore"):
        ra[...], rb[...] = a * c - b * s, b * c + a * s
    return x


def rotate(x, table, pos, interleaved=False):
    """x [rows, heads, 128] rotated by float32 table [positions, dim] (cos, then sin), in float64."""
    return _turn(x, table, pos, interleaved, np.float64)


def rotate32(x, table, pos, interleaved=False):
    """The same with every product and sum rounded to float32."""
    return _turn(x, table, pos, interleaved, np.float32)


def encode(x) -> np.ndarray:
    """Codes (a byte each) of values already divided by their scale: the nearest e2m1 value, ties to the even code."""
    x = np.asarray(x, np.float64)
    size = np.minimum(np.abs(x), 6.0)
    d = np.abs(size[..., None] - E2M1[:8])
    best = d.min(-1, keepdims=True)
    near = d == best
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1, keepdims=True), even, near)
    return (pick.argmax(-1) | (np.signbit(x) << 3)).astype(np.uint8)


def two_a_byte(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def values(packed):
    """float64 values of packed codes."""
    return np.stack([E2M1[packed & 15], E2M1[packed >> 4]], -1).reshape(*packed.shape[:-1], 2 * packed.shape[-1])


def block_exponent(x) -> int:
    x = np.abs(np.asarray(x, np.float64))
    x = x[np.isfinite(x)]
    top = float(x.max()) if x.size else 0.0
    e = LOW
    while e < HIGH and 6.0 * 2.0 ** e < top:
        e += 1
    return e


def quantise_k(x):
    """(packed codes [64], scale bytes [4]) of one head x [128]."""
    codes, scales = np.zeros(128, np.uint8), np.zeros(4, np.uint8)
    for j in range(4):
        b = np.asarray(x[32 * j:32 * j + 32], np.float64)
        e = block_exponent(b)
        codes[32 * j:32 * j + 32] = encode(np.nan_to_num(b, nan=0.0, posinf=np.inf, neginf=-np.inf) / 2.0 ** e)
        scales[j] = NAN_SCALE if np.isnan(b).any() else e + 127
    return two_a_byte(codes), scales


def _bf16(x) -> float:
    m, e = np.frexp(x)
    return float(np.ldexp(np.rint(np.ldexp(m, 8)), int(e) - 8))     # np.rint: ties to even; normal values only


def quantise_v(x):
    """(packed codes [64], bf16 scale as float) of one head x [128]."""
    x = np.asarray(x, np.float64)
    fin = np.abs(x[np.isfinite(x)])
    s = _bf16(max((float(fin.max()) if fin.size else 0.0) / 6.0, 2.0 ** -126))
    codes = encode(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf) / s)
    return two_a_byte(codes), float("nan") if np.isnan(x).any() else s


def append(cache, table, seq_lens, starts, k, v):
    """cache: dict of k, v (packed codes), ks (bytes), vs (float64); returns a copy with rows k, v [rows, heads, 128] appended."""
    cache = {n: np.array(x) for n, x in cache.items()}
    pages, heads, P, _ = cache["k"].shape
    for b, L in enumerate(int(x) for x in seq_lens):
        n = int(starts[b + 1] - starts[b])
        if n <= 0 or L < n or starts[b] < 0 or starts[b + 1] > k.shape[0]:
            continue
        for i in range(n):
            pos, r = L - n + i, int(starts[b]) + i
            page = int(table[b, pos // P]) if pos // P < table.shape[1] else -1
            if not 0 <= page < pages:
                continue
            for h in range(heads):
                cache["k"][page, h, pos % P], cache["ks"][page, h, pos % P] = quantise_k(k[r, h])
                cache["v"][page, h, pos % P], cache["vs"][page, h, pos % P] = quantise_v(v[r, h])
    return cache


def attention(cache, table, seq_lens, starts, q, scale, softcap=0.0, slopes=None, prefix=None):
    """As dense_oracle.attention: out, lse, and A, C, Z for the error bounds.  Rows behind the last request's are NaN."""
    pages, heads, P, _ = cache["k"].shape
    q = np.asarray(q, np.float64)
    rows, q_heads = q.shape[:2]
    g = q_heads // heads
    out, A, C = (np.full((rows, q_heads, 128), np.nan) for _ in range(3))
    lse, Z = (np.full((rows, q_heads), np.nan) for _ in range(2))
    for b, L in enumerate(int(v) for v in seq_lens):
        n = int(starts[b + 1] - starts[b])
        if n <= 0:
            continue
        s = np.arange(L)
        ids = np.array([table[b, i // P] if i // P < table.shape[1] else -1 for i in range(L)], np.int64)
        there = (ids >= 0) & (ids < pages)
        safe = np.where(there, ids, 0)
        pos = L - n + np.arange(n)
        last = pos if prefix is None else np.maximum(pos, min(int(prefix[b]), L) - 1)
        see = there[None] & (s[None] <= last[:, None])                           # [n, L]
        r0 = int(starts[b])
        for h in range(heads):
            ks = np.where(cache["ks"][safe, h, s % P] == NAN_SCALE, np.nan, np.exp2(cache["ks"][safe, h, s % P].astype(np.float64) - 127))
            k = values(cache["k"][safe, h, s % P]) * np.repeat(ks, 32, -1)
            vc, vs = values(cache["v"][safe, h, s % P]), np.asarray(cache["vs"], np.float64)[safe, h, s % P][:, None]
            for head in range(h * g, (h + 1) * g):
                with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
                    z = scale * (q[r0:r0 + n, head] @ k.T)
                    if softcap:
                        z = softcap * np.tanh(z / softcap)
                    if slopes is not None:
                        z = z - float(slopes[head]) * np.abs(pos[:, None] - s[None])
                    for i in range(n):
                        r, m = r0 + i, see[i]
                        if not m.any():
                            out[r, head], lse[r, head], A[r, head], C[r, head], Z[r, head] = 0.0, -np.inf, 0.0, 0.0, 0.0
                            continue
                        zi = z[i, m]
                        top = zi.max()
                        p = np.exp(zi - top)
                        total = p.sum()
                        p = p / total
                        out[r, head] = p @ (vc[m] * vs[m])
                        lse[r, head] = top + np.log(total)
                        A[r, head] = p @ np.abs(vc[m] * vs[m])
                        C[r, head] = p.max() * np.abs(vs[m]).max() * np.abs(vc[m]).sum(0)
                        Z[r, head] = scale * (np.abs(k[m][p > 1e-9]) @ np.abs(q[r, head])).max(initial=0.0)
    return out, lse, A, C, Z
