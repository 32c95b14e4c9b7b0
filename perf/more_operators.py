"""Cases of the rotating K/V appends (4-bit and 8-bit caches) and of the dense paged attention over the 4-bit cache.

Each case names one operator (`op`), its batch and its layout.  A batch is described by the tokens that its requests hold
before the step (`ctx_lo` .. `ctx_hi`, spread evenly) and by how many new tokens they bring (`rows`):
  "decode"    one token each
  "verify:n"  n tokens each (a target token and its drafts)
  "chunk:n"   n tokens each (a piece of a prompt)
  "mixed:n"   one request in eight brings n, one in eight none, some 4, the others one: continuous batching
Head width is 128.  The 4-bit cache:
  codes   [pages, kv_heads, page, 64] bytes of two e2m1 codes each (dims 2i in the low and 2i + 1 in the high half)
  K       one power of two per token, head and 32 dims: [pages, kv_heads, page, 4] bytes, exponent + 127 (255: NaN)
  V       one bfloat16 per token and head: [pages, kv_heads, page]
The 8-bit cache is that of operators.py: e4m3 codes with a float32 scale per page and head.
"""
import math
import random

import torch

own = False

DIM = 128
# e2m1 codes 0 .. 15 and, of magnitudes, the values halfway between neighbours (even: whether a tie goes up)
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
HALFWAY = [(0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)]
LOW, HIGH = -15, 13                                             # exponents of K's scales


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def _append(name, bits, B, lo, hi, rows, P, kv, group, rot, pairs=False):
    return {"name": name, "op": "append", "bits": bits, "B": B, "ctx_lo": lo, "ctx_hi": hi, "rows": rows, "P": P, "kv": kv,
            "group": group, "rot": rot, "pairs": pairs}


def _attend(name, B, lo, hi, rows, P, kv, group, cap=0.0, slopes=False, prefix=0):
    return {"name": name, "op": "attend", "B": B, "ctx_lo": lo, "ctx_hi": hi, "rows": rows, "P": P, "kv": kv, "group": group,
            "cap": cap, "slopes": slopes, "prefix": prefix}


def listed():
    return [
        # a small decode batch, half of each head rotated: latency
        _append("append4_decode_b8", 4, 8, 300, 8192, "decode", 64, 4, 8, 64),
        # a large decode batch at long contexts into the 8-bit cache
        _append("append8_decode_b64", 8, 64, 16384, 131072, "decode", 64, 4, 8, 128),
        # continuous batch with odd lengths, small pages, neighbouring dims rotated together
        _append("append4_mixed_b48", 4, 48, 1, 5000, "mixed:333", 16, 8, 6, 64, True),
        # prompts of 4,096 new tokens in each of 4 requests, 4-bit cache
        _append("append4_prompt_4x4096", 4, 4, 61440, 61440, "chunk:4096", 128, 8, 8, 128),
        # a piece of a prompt, 8-bit cache
        _append("append8_prompt_2x1633", 8, 2, 5, 1000, "chunk:1633", 64, 4, 16, 96),
        # one request with a short context: latency
        _attend("attend4_decode_b1_300", 1, 299, 299, "decode", 64, 4, 8),
        # decode batch of 32 at 8,192 tokens
        _attend("attend4_decode_b32_8k", 32, 8191, 8191, "decode", 64, 4, 8),
        # decode batch of 64 at 16K to 128K tokens
        _attend("attend4_decode_b64_128k", 64, 16383, 131071, "decode", 64, 4, 8),
        # speculative verify: 8 requests, 4 rows each, 240,000 tokens
        _attend("attend4_verify_b8x4_240k", 8, 239996, 239996, "verify:4", 64, 4, 8),
        # a prompt's piece: 4,096 new tokens after 61,440
        _attend("attend4_prompt_4096", 1, 61440, 61440, "chunk:4096", 128, 4, 8),
        # whole prompts of an odd length, many query heads a K/V head
        _attend("attend4_prompt_2x1633", 2, 0, 0, "chunk:1633", 64, 4, 16),
        # continuous batch, capped scores with a distance bias and a prefix that all rows see
        _attend("attend4_mixed_b16_capped", 16, 3, 9001, "mixed:517", 32, 2, 6, cap=30.0, slopes=True, prefix=700),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        kind, n = rng.choice([("decode", 1), ("verify", rng.randint(2, 8)), ("chunk", _log(rng, 2, 4096)), ("mixed", _log(rng, 5, 2000))])
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 5, 6, 8, 12, 16])
        B = _log(rng, 1, max(1, min(256, 1_000_000 // (n * kv * group), 16384 // n)))
        lo = rng.randint(0, 500)
        c = _append("", rng.choice([4, 4, 8]), B, lo, lo + _log(rng, 1, 20000), kind if n == 1 else "%s:%d" % (kind, n), rng.choice([16, 32, 64, 128]),
                    kv, group, rng.choice([32, 64, 64, 96, 128, 128]), rng.random() < 0.4)
    else:
        kind, n = rng.choice([("decode", 1), ("decode", 1), ("verify", rng.randint(2, 8)), ("chunk", _log(rng, 9, 2048)), ("mixed", _log(rng, 5, 700))])
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 6, 8, 12, 16])
        # tokens of the longest request, bounded by the work of the largest listed case (and by what the plain form holds)
        most = 20_000_000 // kv if kind in ("decode", "verify") else 1_200_000_000 // (kv * group * n)
        B = _log(rng, 1, 64 if kind in ("decode", "verify") else 16 if kind == "mixed" else 4)
        hi = _log(rng, 1, max(64, min(200000, most // (B * (n if kind == "verify" else 1)))))
        special = rng.random() < 0.3
        c = _attend("", B, rng.randint(0, hi), hi, kind if n == 1 else "%s:%d" % (kind, n), rng.choice([16, 32, 64, 128]), kv, group,
                    cap=rng.choice([20.0, 50.0]) if special and rng.random() < 0.7 else 0.0, slopes=special and rng.random() < 0.7,
                    prefix=_log(rng, 1, 2000) if special and rng.random() < 0.5 else 0)
    del c["name"]
    return c


def _lengths(case):
    """(tokens held before the step, new tokens) of each request, in the case's own order."""
    B, lo, hi = case["B"], case["ctx_lo"], case["ctx_hi"]
    ctx = [lo + (hi - lo) * i // max(1, B - 1) for i in range(B)]
    kind, _, n = case["rows"].partition(":")
    n = int(n or 1)
    if kind == "mixed":
        new = [n if i % 8 == 0 else 0 if i % 8 == 5 else 4 if i % 3 == 0 else 1 for i in range(B)]
    else:
        new = [n] * B
    return list(zip(ctx, new))


def _pages(tokens, P):
    return -(-tokens // P)


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _nearest(x):
    """The e2m1 codes (bytes of one each) nearest to x, ties to the even code; the largest from 5 on."""
    a = x.abs()
    code = torch.zeros(x.shape, dtype=torch.uint8, device=x.device)
    for at, up in HALFWAY:
        code += a >= at if up else a > at
    return code | (torch.signbit(x).to(torch.uint8) << 3)


def _two_a_byte(codes):
    return codes[..., 0::2] | codes[..., 1::2] << 4


def _quantise_k(x):
    """Codes and scale bytes of float32 x [.., 128]: 2^e, the smallest power of two that takes a block's largest to 6 at most."""
    b = x.unflatten(-1, (4, 32))
    finite = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1)
    m, e = torch.frexp(finite)                                 # finite = m * 2^e, m in [0.5, 1); 6 = 0.75 * 2^3
    e = torch.where(finite > 0, e - torch.where(m > 0.75, 2, 3), LOW).clamp(LOW, HIGH)
    codes = _nearest(b / torch.exp2(e.float())[..., None])
    scales = torch.where(torch.isnan(b).any(-1), 255, e + 127).to(torch.uint8)
    return _two_a_byte(codes.flatten(-2)), scales


def _quantise_v(x):
    """Codes and bfloat16 scales (a sixth of the largest) of float32 x [.., 128]."""
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    s = torch.div(top, torch.full_like(top, 6.0)).clamp(min=2.0 ** -126).to(torch.bfloat16)
    codes = _nearest(x / s.float()[..., None])
    return _two_a_byte(codes), torch.where(torch.isnan(x).any(-1), math.nan, s.float()).to(torch.bfloat16)


def _cache4(n, kv, P, gen):
    """A 4-bit pool as appends leave it: normal values, tokens of differing magnitude, some dims of K larger than the others."""
    k_codes = torch.empty((n, kv, P, DIM // 2), dtype=torch.uint8, device="cuda")
    v_codes = torch.empty_like(k_codes)
    k_scales = torch.empty((n, kv, P, 4), dtype=torch.uint8, device="cuda")
    v_scales = torch.empty((n, kv, P), dtype=torch.bfloat16, device="cuda")
    wide = torch.where(torch.rand((kv, 1, DIM), device="cuda", generator=gen) < 1 / 16, 4.0, 0.8)
    step = max(1, (1 << 28) // (kv * P * DIM))
    for i in range(0, n, step):
        m = min(step, n - i)
        size = torch.exp2(0.5 * torch.randn((m, kv, P, 1), device="cuda", generator=gen))
        k_codes[i:i + m], k_scales[i:i + m] = _quantise_k(torch.randn((m, kv, P, DIM), device="cuda", generator=gen) * wide)
        v_codes[i:i + m], v_scales[i:i + m] = _quantise_v(torch.randn((m, kv, P, DIM), device="cuda", generator=gen) * size)
    return k_codes, v_codes, k_scales, v_scales


def _cache8(n, kv, P, gen):
    """An 8-bit pool: power-of-two scales, pages of differing magnitude."""
    codes = [torch.randint(0, 120, (n, kv, P, DIM), dtype=torch.uint8, device="cuda", generator=gen) for _ in "kv"]
    scales = [torch.exp2(torch.randint(-9, -5, (n, kv), device="cuda", generator=gen).float()) for _ in "kv"]
    return codes[0], codes[1], scales[0], scales[1]


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens, P, B, kv = _lengths(case), case["P"], case["B"], case["kv"]
    rng.shuffle(lens)                      # the requests' order
    rows = sum(n for _, n in lens)
    most = max(c + n for c, n in lens)
    width = _pages(most, P) + 3
    held = [_pages(c + n, P) for c, n in lens]
    total = sum(held) + 5
    perm = torch.randperm(total, device="cuda", generator=gen).to(torch.int32)
    at = torch.arange(width, device="cuda")[None]
    start = torch.tensor([0] + held[:-1], device="cuda").cumsum(0)[:, None]
    table = torch.where(at < torch.tensor(held, device="cuda")[:, None], perm[(start + at).clamp(max=total - 1)], -1).to(torch.int32)
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    heads = kv * case["group"]
    st = {"op": case["op"], "P": P, "kv": kv, "rows": rows, "most": most, "most_new": max(n for _, n in lens), "table": table,
          "seq_lens": _int32([c + n for c, n in lens]), "starts": _int32(starts), "bits": case.get("bits", 4)}
    st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"] = (_cache4 if st["bits"] == 4 else _cache8)(total, kv, P, gen)
    if case["op"] == "append":
        # q, k and v as one projection leaves them; a token in 16 is an outlier
        qkv = torch.randn((rows, heads + 2 * kv, DIM), device="cuda", generator=gen)
        qkv *= torch.where(torch.rand((rows, 1, 1), device="cuda", generator=gen) < 1 / 16, 6.0, 1.0)
        qkv = qkv.to(torch.bfloat16)
        st["q"], st["k"], st["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        st["q_out"] = torch.empty((rows, heads, DIM), dtype=torch.bfloat16, device="cuda")   # a serving loop keeps it
        st["rot"], st["pairs"] = case["rot"], case["pairs"]
        # cos and sin of every position, made once for a model
        turn = torch.arange(most, device="cuda").double()[:, None] * 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda").double() / case["rot"])
        st["table_cs"] = torch.cat([turn.cos(), turn.sin()], 1).float()
        return st
    st["q"] = torch.randn((rows, heads, DIM), device="cuda", generator=gen).to(torch.bfloat16)
    st["scale"] = DIM ** -0.5
    st["cap"] = case["cap"]
    st["slopes"] = torch.exp2(-8.0 * (torch.arange(heads, device="cuda") + 1) / heads).to(torch.float32) if case["slopes"] else None
    st["prefix"] = _int32([min(case["prefix"], c + n) for c, n in lens]) if case["prefix"] else None
    return st


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------
def run(state):
    return (_run_append if state["op"] == "append" else _run_attend)(state)


def _handles(st):
    """The framework's objects over the state's tensors: a program makes them once for a cache, a batch and a model."""
    if "handles" not in st:
        import deepseek_sparse_mla_gb300 as dsa
        cache = (dsa.Kv4Cache if st["bits"] == 4 else dsa.BlockKvCache).of(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"])
        batch = dsa.Batch(st["table"], st["seq_lens"], st["starts"], num_rows=st["rows"], max_seq_len=st["most"])
        rope = dsa.RotaryTable.of(st["table_cs"], interleaved=st["pairs"]) if st["op"] == "append" else None
        st["handles"] = dsa, cache, batch, rope
    return st["handles"]


def _rotated(x, pos, table, rot, pairs):
    """float32 x [rows, heads, 128] with its first `rot` dims rotated by their positions' angles."""
    c, s = table[pos][:, None].chunk(2, -1)
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _places(st):
    """Request and position of each row."""
    starts, lens = st["starts"].long(), st["seq_lens"].long()
    t = torch.arange(st["rows"], device="cuda")
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    return b, lens[b] - starts[b + 1] + t


# 4-bit codes come back as the bytes that hold two of them: nothing in them is a matter of rounding errors, as the
# rotation's products and difference are each rounded to float32 and every quotient is exact or IEEE's.
def _run_append(st):
    if own:
        dsa, cache, batch, rope = _handles(st)
        append = dsa.kv4_append if st["bits"] == 4 else dsa.kv8_append
        append(cache, batch, st["k"], st["v"], rope=rope, q=st["q"], q_out=st["q_out"])
        q = st["q_out"]
    else:
        b, pos = _places(st)
        k = _rotated(st["k"], pos, st["table_cs"], st["rot"], st["pairs"])
        q = _rotated(st["q"], pos, st["table_cs"], st["rot"], st["pairs"]).to(torch.bfloat16)
        if st["bits"] == 8:
            _pages8(st, k)
        else:
            page, off = st["table"][b, pos // st["P"]].long()[:, None], (pos % st["P"])[:, None]
            at = page, torch.arange(st["kv"], device="cuda")[None], off
            st["k_codes"][at], st["k_scales"][at] = _quantise_k(k)
            st["v_codes"][at], st["v_scales"][at] = _quantise_v(st["v"].float())
    if st["bits"] == 8:
        return {"k": st["k_codes"].view(torch.float8_e4m3fn), "v": st["v_codes"].view(torch.float8_e4m3fn), "k_scales": st["k_scales"],
                "v_scales": st["v_scales"], "q": q}
    return {"k": st["k_codes"], "v": st["v_codes"], "k_scales": st["k_scales"], "v_scales": st["v_scales"], "q": q}


def _pages8(st, k):
    """The 8-bit append of rotated k: a page whose new tokens need a larger scale is coded again."""
    P, T, B = st["P"], st["rows"], st["seq_lens"].shape[0]
    starts, lens = st["starts"].long(), st["seq_lens"].long()
    new = starts[1:] - starts[:-1]
    first = (lens - new) // P                                  # the first page that a request writes
    count = torch.where(new > 0, (lens - 1) // P - first + 1, 0)
    ends = count.cumsum(0)
    u = torch.arange(T // P + 2 * B, device="cuda")            # as many pages as the step can touch; the last one again past the end
    u = torch.minimum(u, ends[-1] - 1)
    b = torch.searchsorted(ends, u, right=True)
    lp = first[b] + u - (ends[b] - count[b])
    page = st["table"][b, lp.clamp(0, st["table"].shape[1] - 1)].long().clamp(min=0)
    pos = lp[:, None] * P + torch.arange(P, device="cuda")
    i = pos - (lens - new)[b][:, None]                         # which of the request's new tokens
    is_new, is_old = (i >= 0) & (i < new[b][:, None]), i < 0
    row = (starts[b][:, None] + i).clamp(0, T - 1)
    for codes, scales, x in ((st["k_codes"], st["k_scales"], k), (st["v_codes"], st["v_scales"], st["v"])):
        fresh = x[row].float() * is_new[..., None, None]       # [pages, P, kv, 128]
        m, e = torch.frexp(fresh.abs().amax((1, 3)))           # 448 = 0.875 * 2^9
        want = torch.where(m > 0, torch.exp2((e - torch.where(m > 0.875, 8, 9)).float()), 2.0 ** -126)
        have = torch.where(is_old.any(1)[:, None], scales[page], 0.0)
        s = torch.maximum(want, have)
        held = codes[page].view(torch.float8_e4m3fn).float().transpose(1, 2) * (scales[page] / s)[:, None, :, None]
        fresh = (fresh / s[:, None, :, None]).clamp(-448.0, 448.0)
        change = is_new[:, :, None] | (is_old[:, :, None] & (have < s)[:, None])
        both = torch.where(is_new[..., None, None], fresh, held)
        q = torch.where(change[..., None], both.to(torch.float8_e4m3fn).view(torch.uint8), codes[page].transpose(1, 2)).transpose(1, 2)
        codes[page], scales[page] = q, s


def _values(codes, dtype):
    """Values of bytes of two e2m1 codes each."""
    one = torch.tensor(E2M1 + [-v for v in E2M1], dtype=dtype, device="cuda")
    both = torch.stack([one.repeat(16), one.repeat_interleave(16)], -1)          # of each byte: low half, high half
    return both[codes.int()].flatten(-2)


def _run_attend(st):
    if own:
        dsa, cache, batch, _ = _handles(st)
        return dsa.paged_attention(cache, batch, st["q"], st["scale"], max_query_len=st["most_new"], softcap=st["cap"], slopes=st["slopes"],
                                   prefix_lens=st["prefix"])[0]
    P, kv, T, N = st["P"], st["kv"], st["rows"], st["most_new"]
    starts, lens = st["starts"].long(), st["seq_lens"].long()
    B, heads = lens.shape[0], st["q"].shape[1]
    g = heads // kv
    pages = st["table"][:, : _pages(st["most"], P)].long().clamp(min=0)
    S = pages.shape[1] * P

    def tokens(x):
        return x.transpose(1, 2).reshape(B, kv, S, DIM)

    def keys():
        k = _values(st["k_codes"][pages], torch.float32)
        k.unflatten(-1, (4, 32)).mul_(torch.exp2(st["k_scales"][pages].float() - 127.0)[..., None])
        return tokens(k)

    i = torch.arange(N, device="cuda")
    new = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + i).clamp(max=T - 1)                                            # [B, N]
    q = st["q"][row].float().view(B, N, kv, g, DIM).permute(0, 2, 3, 1, 4).reshape(B, kv, g * N, DIM)
    z = (q @ keys().transpose(2, 3)).mul_(st["scale"]).view(B, kv, g, N, S)
    if st["cap"]:
        z = z.div_(st["cap"]).tanh_().mul_(st["cap"])
    pos = (lens - new)[:, None] + i                                                            # [B, N]
    j = torch.arange(S, device="cuda")
    if st["slopes"] is not None:
        away = (pos[..., None] - j).abs_().float()
        z -= st["slopes"].view(kv, g, 1, 1) * away[:, None, None]
    last = pos if st["prefix"] is None else torch.maximum(pos, torch.minimum(st["prefix"].long(), lens)[:, None] - 1)
    z.masked_fill_((j > last[..., None])[:, None, None], -math.inf)
    z = z.sub_(z.amax(-1, keepdim=True)).exp_()
    total = z.sum(-1, keepdim=True)
    v = tokens(_values(st["v_codes"][pages], torch.float32).mul_(st["v_scales"][pages].float()[..., None]))
    o = (z.view(B, kv, g * N, S) @ v).view(B, kv, g, N, DIM) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, heads, DIM)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    return o[b, t - starts[b]].to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    lens, P, kv = _lengths(case), case["P"], case["kv"]
    rows, heads = sum(n for _, n in lens), case["kv"] * case["group"]
    if case["op"] == "append":
        # q in and out, k and v in; the codes, with their scales; a row of cos and sin and a page id a token
        codes = kv * (2 * DIM if case["bits"] == 8 else DIM + 6)
        touched = sum(_pages(c + n, P) - c // P for c, n in lens if n)
        return {"bytes": float(rows * (4 * heads * DIM + 4 * kv * DIM + codes + 4 * case["rot"]) + touched * (4 + (16 * kv if case["bits"] == 8 else 0))),
                "flops": 3.0 * rows * (heads + kv) * case["rot"]}
    held = sum(c + n for c, n in lens if n)
    seen = 0
    for c, n in lens:
        p = min(case["prefix"], c + n)
        seen += sum(max(c + i + 1, p) for i in range(n))
    return {"bytes": held * kv * (DIM + 6.0) + 4.0 * rows * heads * DIM, "flops": 4.0 * heads * DIM * seen}


# ---------------------------------------------------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(st) if st["op"] == "append" else _exact_attend(st, case)


def _e4m3(x):
    """The nearest e4m3 value of each of x (float64, at most 448 in size), ties to the even code."""
    _, e = torch.frexp(x)
    step = ((e - 4).clamp(min=-9).long() + 1023 << 52).view(torch.float64)      # 2^(e - 4): 4 significant bits, subnormal steps of 2^-9
    return torch.round(x / step) * step


def _exact_append(st):
    """Rotated q and the scales; e4m3 values of the 8-bit cache.  (Bytes of 4-bit codes are whole numbers.)"""
    P, starts, lens, table = st["P"], st["starts"].tolist(), st["seq_lens"].tolist(), st["table"].tolist()
    rot, half = st["rot"], st["rot"] // 2
    place = [(b, lens[b] - starts[b + 1] + r) for b in range(len(lens)) for r in range(starts[b], starts[b + 1])]
    angle = st["table_cs"].double()[torch.tensor([p for _, p in place], device="cuda")]
    turn = torch.complex(angle[:, :half], angle[:, half:])[:, None]

    def rotate(x):
        x = x.double()
        z = (torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) if st["pairs"] else torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous())) * turn
        out = x.clone()
        if st["pairs"]:
            out[..., 0:rot:2], out[..., 1:rot:2] = z.real, z.imag
        else:
            out[..., :half], out[..., half:rot] = z.real, z.imag
        return out

    k, v = rotate(st["k"]), st["v"].double()
    if st["bits"] == 4:
        at = (torch.tensor([table[b][p // P] for b, p in place], device="cuda")[:, None], torch.arange(st["kv"], device="cuda")[None],
              torch.tensor([p % P for _, p in place], device="cuda")[:, None])
        scales = st["v_scales"].double()
        scales[at] = (v.abs().amax(-1) / 6).clamp(min=2.0 ** -126).to(torch.bfloat16).double()
        return {"k": None, "v": None, "k_scales": None, "v_scales": scales, "q": rotate(st["q"])}
    out = {"q": rotate(st["q"])}
    for name, x in (("k", k), ("v", v)):
        value = st[name + "_codes"].view(torch.float8_e4m3fn).double()
        scale = st[name + "_scales"].double()
        for b, L in enumerate(lens):
            at, end = L - (starts[b + 1] - starts[b]), L
            r = starts[b]
            while at < end:
                page, off = table[b][at // P], at % P
                n = min(P - off, end - at)
                rows = x[r:r + n].transpose(0, 1)                      # [kv, n, 128]
                top = rows.abs().amax((1, 2))
                want = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
                want = torch.where(top > 0, torch.where(top > 448.0 * want, 2 * want, torch.where(2 * top <= 448.0 * want, want / 2, want)), 2.0 ** -126)
                s = torch.maximum(want, scale[page]) if off else want
                if off:
                    value[page, :, :off] = _e4m3(value[page, :, :off] * (scale[page] / s)[:, None, None])
                value[page, :, off:off + n] = _e4m3(rows / s[:, None, None])
                scale[page] = s
                at, r = at + n, r + n
        out[name], out[name + "_scales"] = value, scale
    return out


def _exact_attend(st, case):
    if work(case)["flops"] > 6e12:
        return None
    P, kv = st["P"], st["kv"]
    starts, lens = st["starts"].tolist(), st["seq_lens"].tolist()
    heads = st["q"].shape[1]
    g = heads // kv
    out = torch.zeros((st["rows"], heads, DIM), dtype=torch.float64, device="cuda")
    size = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

    def value(byte):
        halves = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).int()
        return torch.where(halves > 7, -1.0, 1.0) * size[halves & 7]

    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        if not n:
            continue
        pages = st["table"][b, : _pages(L, P)].long()
        for h in range(kv):
            k = value(st["k_codes"][pages, h]) * torch.exp2(st["k_scales"][pages, h].double() - 127).repeat_interleave(32, -1)
            v = value(st["v_codes"][pages, h]) * st["v_scales"][pages, h].double()[..., None]
            k, v = k.view(-1, DIM)[:L], v.view(-1, DIM)[:L]
            j = torch.arange(L, device="cuda", dtype=torch.float64)
            step = max(1, (1 << 27) // (g * L))
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                q = st["q"][starts[b] + i0:starts[b] + i1, h * g:(h + 1) * g].double()      # [rows, g, 128]
                z = torch.einsum("ngd,sd->ngs", q, k) * st["scale"]
                if st["cap"]:
                    z = st["cap"] * torch.tanh(z / st["cap"])
                pos = torch.arange(L - n + i0, L - n + i1, device="cuda", dtype=torch.float64)
                if st["slopes"] is not None:
                    z = z - st["slopes"][h * g:(h + 1) * g].double()[None, :, None] * (pos[:, None, None] - j).abs()
                end = pos if st["prefix"] is None else pos.clamp(min=float(min(int(st["prefix"][b]), L) - 1))
                z = torch.where(j <= end[:, None, None], z, -math.inf)
                out[starts[b] + i0:starts[b] + i1, h * g:(h + 1) * g] = torch.einsum("ngs,sd->ngd", torch.softmax(z, -1), v)
    return out
