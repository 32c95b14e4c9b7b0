"""Cases of the step planner, the block-scaled 8-bit K/V append and the dense paged attention over that cache.

Each case names one operator (`op`), its batch and its layout.  A batch is described by the tokens that its requests hold
before the step (`ctx_lo` .. `ctx_hi`, spread evenly) and by how many new tokens they bring (`rows`):
  "decode"    one token each
  "verify:n"  n tokens each (a target token and its drafts)
  "chunk:n"   n tokens each (a piece of a prompt)
  "mixed:n"   one request in eight brings n, one in eight none, some 4, the others one: continuous batching
Head width is 128; K and V are e4m3 codes [pages, kv_heads, page_size, 128] with one float32 scale per page and head.
"""
import math
import random

import torch

own = False

DIM = 128


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def _plan(name, B, lo, hi, rows, P):
    return {"name": name, "op": "plan", "B": B, "ctx_lo": lo, "ctx_hi": hi, "rows": rows, "P": P}


def _append(name, B, lo, hi, rows, P, kv):
    return {"name": name, "op": "append", "B": B, "ctx_lo": lo, "ctx_hi": hi, "rows": rows, "P": P, "kv": kv}


def _attend(name, B, lo, hi, rows, P, kv, group, cap=0.0, slopes=False, prefix=0):
    return {"name": name, "op": "attend", "B": B, "ctx_lo": lo, "ctx_hi": hi, "rows": rows, "P": P, "kv": kv, "group": group,
            "cap": cap, "slopes": slopes, "prefix": prefix}


def listed():
    return [
        # a small decode batch's step: latency
        _plan("plan_decode_b8", 8, 300, 8192, "decode", 64),
        # a continuous batch: decode rows, verify rows, prompt pieces, idle requests
        _plan("plan_mixed_b256", 256, 0, 131072, "mixed:197", 64),
        # a large scheduler step over thousands of requests with a small page
        _plan("plan_chunks_b4096", 4096, 5, 16384, "chunk:17", 16),
        # decode batch's append: one token a request, most pages keep their scale
        _append("append_decode_b64", 64, 16384, 131072, "decode", 64, 4),
        # continuous batch with odd lengths and small pages
        _append("append_mixed_b48", 48, 1, 5000, "mixed:333", 16, 8),
        # a prompt of 4,096 new tokens in each of 4 requests
        _append("append_prompt_4x4096", 4, 61440, 61440, "chunk:4096", 128, 8),
        # one request with a short context: latency
        _attend("attend_decode_b1_300", 1, 299, 299, "decode", 64, 4, 8),
        # decode batch of 32 at 8,192 tokens
        _attend("attend_decode_b32_8k", 32, 8191, 8191, "decode", 64, 4, 8),
        # decode batch of 64 at 16K to 128K tokens
        _attend("attend_decode_b64_128k", 64, 16383, 131071, "decode", 64, 4, 8),
        # speculative verify: 8 requests, 4 rows each, 240,000 tokens
        _attend("attend_verify_b8x4_240k", 8, 239996, 239996, "verify:4", 64, 4, 8),
        # a prompt's piece: 4,096 new tokens after 61,440
        _attend("attend_prompt_4096", 1, 61440, 61440, "chunk:4096", 128, 4, 8),
        # continuous batch, capped scores with a distance bias and a prefix that all rows see
        _attend("attend_mixed_b16_capped", 16, 3, 9001, "mixed:517", 32, 2, 6, cap=30.0, slopes=True, prefix=700),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend"])
    if op == "plan":
        kind, n = rng.choice([("decode", 1), ("verify", rng.randint(2, 8)), ("chunk", _log(rng, 2, 4000)), ("mixed", _log(rng, 5, 4000))])
        B = _log(rng, 1, max(1, min(4096, 69632 // n)))
        lo = rng.randint(0, 500)
        c = _plan("", B, lo, lo + _log(rng, 1, 100000), kind if n == 1 else "%s:%d" % (kind, n), rng.choice([16, 32, 64, 128]))
    elif op == "append":
        kind, n = rng.choice([("decode", 1), ("verify", rng.randint(2, 8)), ("chunk", _log(rng, 2, 4096)), ("mixed", _log(rng, 5, 2000))])
        B = _log(rng, 1, max(1, min(256, 16384 // n)))
        lo = rng.randint(0, 500)
        c = _append("", B, lo, lo + _log(rng, 1, 20000), kind if n == 1 else "%s:%d" % (kind, n), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 8]))
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


def _quantised_pages(n, kv, P, gen):
    """A pool's codes and scales as an append leaves them: normal values, pages of differing magnitude, power-of-two scales."""
    codes = torch.empty((n, kv, P, DIM), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, kv), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 28) // (kv * P * DIM))
    for i in range(0, n, step):
        m = min(step, n - i)
        x = torch.randn((m, kv, P, DIM), device="cuda", generator=gen)
        x *= torch.exp2(0.5 * torch.randn((m, kv, 1, 1), device="cuda", generator=gen))
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448.0)))
        x /= s[..., None, None]
        codes[i:i + m] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        scales[i:i + m] = s
    return codes, scales


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens, P, B = _lengths(case), case["P"], case["B"]
    rng.shuffle(lens)                      # the requests' order
    rows = sum(n for _, n in lens)
    most = max(c + n for c, n in lens)
    width = _pages(most, P) + 3
    if case["op"] == "plan":
        held = [_pages(c, P) for c, _ in lens]
        taken = sum(held)
        need = sum(_pages(c + n, P) for c, n in lens) - taken
        total = taken + need + 57
        perm = torch.randperm(total, device="cuda", generator=gen).to(torch.int32)
        width = -(-width // 8) * 8
        at = torch.arange(width, device="cuda")[None]
        start = torch.tensor([0] + held[:-1], device="cuda").cumsum(0)[:, None]
        table = torch.where(at < torch.tensor(held, device="cuda")[:, None], perm[(start + at).clamp(max=total - 1)], -1).to(torch.int32)
        free = torch.zeros(total, dtype=torch.int32, device="cuda")
        free[:need + 57] = perm[taken:]
        return {"op": "plan", "P": P, "rows": rows, "seq_lens": _int32([c for c, _ in lens]), "new_lens": _int32([n for _, n in lens]),
                "table": table, "free": free, "count": _int32([need + 57]),
                # the buffers of a step that a serving loop keeps
                "seq_lens_out": torch.zeros(B, dtype=torch.int32, device="cuda"), "starts": torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
                "slots": torch.zeros(rows, dtype=torch.int64, device="cuda"), "positions": torch.zeros(rows, dtype=torch.int32, device="cuda"),
                "count_out": _int32([0])}
    held = [_pages(c + n, P) for c, n in lens]
    total = sum(held) + 5
    perm = torch.randperm(total, device="cuda", generator=gen).to(torch.int32)
    at = torch.arange(width, device="cuda")[None]
    start = torch.tensor([0] + held[:-1], device="cuda").cumsum(0)[:, None]
    table = torch.where(at < torch.tensor(held, device="cuda")[:, None], perm[(start + at).clamp(max=total - 1)], -1).to(torch.int32)
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    kv = case["kv"]
    st = {"op": case["op"], "P": P, "kv": kv, "rows": rows, "most": most, "most_new": max(n for _, n in lens), "table": table,
          "seq_lens": _int32([c + n for c, n in lens]), "starts": _int32(starts)}
    st["k_codes"], st["k_scales"] = _quantised_pages(total, kv, P, gen)
    st["v_codes"], st["v_scales"] = _quantised_pages(total, kv, P, gen)
    if case["op"] == "append":
        # a token in 16 is an outlier, so that some pages need a larger scale than they have
        big = torch.where(torch.rand((rows, 1, 1), device="cuda", generator=gen) < 1 / 16, 6.0, 1.0)
        st["k"] = (torch.randn((rows, kv, DIM), device="cuda", generator=gen) * big).to(torch.bfloat16)
        st["v"] = (torch.randn((rows, kv, DIM), device="cuda", generator=gen) * big).to(torch.bfloat16)
        return st
    heads = kv * case["group"]
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
    return {"plan": _run_plan, "append": _run_append, "attend": _run_attend}[state["op"]](state)


def _handles(st):
    """The framework's objects over the state's tensors: a program makes them once for a cache and a batch."""
    if "handles" not in st:
        import deepseek_sparse_mla_gb300 as dsa
        if st["op"] == "plan":
            st["handles"] = dsa, dsa.PagePool.of(st["free"], st["count"])
        else:
            batch = dsa.Batch(st["table"], st["seq_lens"], st["starts"], num_rows=st["rows"], max_seq_len=st["most"])
            st["handles"] = dsa, dsa.BlockKvCache.of(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"]), batch
    return st["handles"]


def _run_plan(st):
    table, P = st["table"], st["P"]
    if own:
        dsa, pool = _handles(st)
        dsa.step_plan(pool, st["seq_lens"], st["new_lens"], table, P, st["rows"], seq_lens_out=st["seq_lens_out"],
                      query_start_loc=st["starts"], slot_mapping=st["slots"], positions=st["positions"], free_count_out=st["count_out"])
        return {"seq_lens": st["seq_lens_out"], "starts": st["starts"], "slots": st["slots"], "positions": st["positions"],
                "count": st["count_out"], "table": table}
    old, new = st["seq_lens"].long(), st["new_lens"].long()
    held = (old + P - 1) // P
    need = (old + new + P - 1) // P - held
    # the longest run of requests, from the first on, whose pages and rows there are
    fits = (need.cumsum(0) <= st["count"].long()) & (new.cumsum(0) <= st["rows"])
    need, new = need * fits, new * fits
    ends = new.cumsum(0)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    first = need.cumsum(0) - need
    at = torch.arange(table.shape[1], device="cuda")[None] - held[:, None]       # which of the request's new pages
    page = st["free"][(st["count"].long() - 1 - first[:, None] - at).clamp(0, st["free"].shape[0] - 1)]
    table = torch.where((at >= 0) & (at < need[:, None]), page, table)
    r = torch.arange(st["rows"], device="cuda")
    b = torch.searchsorted(ends, r, right=True).clamp(max=old.shape[0] - 1)
    pos = old[b] + r - starts[b]
    slot = table[b, (pos // P).clamp(max=table.shape[1] - 1)].long() * P + pos % P
    live = r < ends[-1]
    return {"seq_lens": (old + new).int(), "starts": starts.int(), "slots": torch.where(live, slot, -1),
            "positions": torch.where(live, pos, -1).int(), "count": (st["count"].long() - need.sum()).int(), "table": table}


def _run_append(st):
    if own:
        dsa, cache, batch = _handles(st)
        dsa.kv8_append(cache, batch, st["k"], st["v"])
    else:
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
        for codes, scales, x in ((st["k_codes"], st["k_scales"], st["k"]), (st["v_codes"], st["v_scales"], st["v"])):
            fresh = x[row].float() * is_new[..., None, None]       # [pages, P, kv, 128]
            m, e = torch.frexp(fresh.abs().amax((1, 3)))           # 448 = 0.875 * 2^9
            want = torch.where(m > 0, torch.exp2((e - torch.where(m > 0.875, 8, 9)).float()), 2.0 ** -126)
            have = torch.where(is_old.any(1)[:, None], scales[page], 0.0)
            s = torch.maximum(want, have)
            held = codes[page].view(torch.float8_e4m3fn).float().transpose(1, 2) * (scales[page] / s)[:, None, :, None]
            fresh = (fresh / s[:, None, :, None]).clamp(-448.0, 448.0)
            all_ = torch.where(is_new[..., None, None], fresh, torch.where((is_old[:, :, None] & (have < s)[:, None])[..., None], held, 0.0))
            change = is_new[:, :, None] | (is_old[:, :, None] & (have < s)[:, None])
            q = torch.where(change[..., None], all_.to(torch.float8_e4m3fn).view(torch.uint8), codes[page].transpose(1, 2)).transpose(1, 2)
            codes[page], scales[page] = q, s
    return {"k": st["k_codes"].view(torch.float8_e4m3fn), "v": st["v_codes"].view(torch.float8_e4m3fn), "k_scales": st["k_scales"], "v_scales": st["v_scales"]}


def _run_attend(st):
    if own:
        dsa, cache, batch = _handles(st)
        return dsa.paged_attention(cache, batch, st["q"], st["scale"], max_query_len=st["most_new"], softcap=st["cap"], slopes=st["slopes"],
                                   prefix_lens=st["prefix"])[0]
    P, kv, T, N = st["P"], st["kv"], st["rows"], st["most_new"]
    starts, lens = st["starts"].long(), st["seq_lens"].long()
    B, heads = lens.shape[0], st["q"].shape[1]
    g = heads // kv
    pages = st["table"][:, : _pages(st["most"], P)].long().clamp(min=0)
    S = pages.shape[1] * P

    def tokens(codes, scales):
        x = codes[pages].view(torch.float8_e4m3fn).float()
        x *= scales[pages][..., None, None]
        return x.transpose(1, 2).reshape(B, kv, S, DIM)

    i = torch.arange(N, device="cuda")
    new = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + i).clamp(max=T - 1)                                            # [B, N]
    q = st["q"][row].float().view(B, N, kv, g, DIM).permute(0, 2, 3, 1, 4).reshape(B, kv, g * N, DIM)
    z = (q @ tokens(st["k_codes"], st["k_scales"]).transpose(2, 3)).mul_(st["scale"]).view(B, kv, g, N, S)
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
    o = (z.view(B, kv, g * N, S) @ tokens(st["v_codes"], st["v_scales"])).view(B, kv, g, N, DIM) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, heads, DIM)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    return o[b, t - starts[b]].to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    lens, P = _lengths(case), case["P"]
    rows, B = sum(n for _, n in lens), case["B"]
    if case["op"] == "plan":
        fresh = sum(_pages(c + n, P) - _pages(c, P) for c, n in lens)
        # lengths in and out, starts; a page id read and written per new page; slot and position per row, and its page's id
        return {"bytes": 16.0 * B + 8.0 * fresh + 12.0 * rows + 4.0 * sum(_pages(n, P) for _, n in lens), "flops": 0.0}
    kv = case["kv"]
    if case["op"] == "append":
        touched = sum(_pages(c + n, P) - c // P for c, n in lens if n)
        return {"bytes": 2.0 * kv * (rows * DIM * 3 + touched * 8) + 4.0 * touched, "flops": 0.0}
    heads = kv * case["group"]
    held = sum(c + n for c, n in lens if n)
    seen = 0
    for c, n in lens:
        p = min(case["prefix"], c + n)
        seen += sum(max(c + i + 1, p) for i in range(n))
    return {"bytes": 2.0 * held * kv * DIM + 2.0 * sum(_pages(c + n, P) for c, n in lens if n) * kv * 4 + 4.0 * rows * heads * DIM,
            "flops": 4.0 * heads * DIM * seen}


# ---------------------------------------------------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "plan":
        return None
    return _exact_append(st) if st["op"] == "append" else _exact_attend(st, case)


def _e4m3(x):
    """The nearest e4m3 value of each of x (float64, at most 448 in size), ties to the even code."""
    _, e = torch.frexp(x)
    step = ((e - 4).clamp(min=-9).long() + 1023 << 52).view(torch.float64)      # 2^(e - 4): 4 significant bits, subnormal steps of 2^-9
    return torch.round(x / step) * step


def _exact_append(st):
    P, starts, lens, table = st["P"], st["starts"].tolist(), st["seq_lens"].tolist(), st["table"].tolist()
    out = {}
    for name in "kv":
        value = st[name + "_codes"].view(torch.float8_e4m3fn).double()
        scale = st[name + "_scales"].double()
        x = st[name].double()
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
    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        if not n:
            continue
        pages = st["table"][b, : _pages(L, P)].long()
        for h in range(kv):
            k = (st["k_codes"][pages, h].view(torch.float8_e4m3fn).double() * st["k_scales"][pages, h].double()[:, None, None]).view(-1, DIM)[:L]
            v = (st["v_codes"][pages, h].view(torch.float8_e4m3fn).double() * st["v_scales"][pages, h].double()[:, None, None]).view(-1, DIM)[:L]
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
