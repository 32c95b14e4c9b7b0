"""The step planner, the 8-bit append and the dense attention reject bad arguments on the host, before any launch (no GPU)."""
import ctypes

import pytest

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
A = 1 << 20                                                 # an aligned address that is never dereferenced


def _cache(**kw):
    from deepseek_sparse_mla_gb300._lib import DsaKv8Cache
    f = dict(k=A, v=A, ks=A, vs=A, pages=16, P=64, heads=2, reserved=0, **{})
    f.update(kw)
    return DsaKv8Cache(f["k"], f["v"], f["ks"], f["vs"], f["pages"], f["P"], f["heads"], f["reserved"])


def _batch(table=A, lens=A, qsl=A, B=2, rows=2, L=300, stride=8):
    from deepseek_sparse_mla_gb300._lib import DsaBatch
    return DsaBatch(table, lens, qsl, B, rows, L, stride)


def _said(lib, status, want, word):
    assert status == want, (status, lib.dsa_last_error())
    assert word in lib.dsa_last_error().decode()


BAD_CACHES = [(dict(k=0), INVALID, "NULL"), (dict(vs=0), INVALID, "NULL"), (dict(v=A + 8), INVALID, "aligned"),
              (dict(ks=A + 2), INVALID, "aligned"), (dict(pages=0), INVALID, "num_pages"), (dict(P=48), UNSUPPORTED, "page_size"),
              (dict(P=256), UNSUPPORTED, "page_size"), (dict(P=8), UNSUPPORTED, "page_size"), (dict(heads=0), INVALID, "kv_heads"),
              (dict(pages=1 << 30), UNSUPPORTED, "2^31"), (dict(reserved=1), INVALID, "reserved")]
BAD_BATCHES = [(dict(table=0), INVALID, "NULL"), (dict(lens=0), INVALID, "NULL"), (dict(B=0), INVALID, "num_requests"),
               (dict(rows=-1), INVALID, "num_rows"), (dict(stride=0), INVALID, "block_table_stride"),
               (dict(qsl=0, rows=5), INVALID, "num_rows")]


def _append(lib, cache=None, batch=None, k=A, ks=256, v=A, vs=256):
    return lib.dsa_kv8_append(ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()), k, ks, v, vs, None)


@pytest.mark.parametrize("kw,status,word", BAD_CACHES)
def test_append_rejects_bad_caches(lib, kw, status, word):
    _said(lib, _append(lib, cache=_cache(**kw)), status, word)


@pytest.mark.parametrize("kw,status,word", BAD_BATCHES)
def test_append_rejects_bad_batches(lib, kw, status, word):
    _said(lib, _append(lib, batch=_batch(**kw)), status, word)


@pytest.mark.parametrize("kw,word", [(dict(k=0), "k is NULL"), (dict(v=0), "v is NULL"), (dict(k=A + 2), "aligned"),
                                     (dict(ks=255), "stride"), (dict(vs=128), "stride"), (dict(vs=260), "stride")])
def test_append_rejects_bad_rows(lib, kw, word):
    _said(lib, _append(lib, **kw), INVALID, word)


def test_null_structs_and_calls_without_rows(lib):
    b, c = _batch(), _cache()
    _said(lib, lib.dsa_kv8_append(None, ctypes.byref(b), A, 256, A, 256, None), INVALID, "cache is NULL")
    _said(lib, lib.dsa_kv8_append(ctypes.byref(c), None, A, 256, A, 256, None), INVALID, "batch is NULL")
    _said(lib, lib.dsa_paged_attention(None, ctypes.byref(b), A, 512, 4, 1.0, 1, None, A, None, A, 1 << 30, None), INVALID, "cache")
    assert _append(lib, batch=_batch(rows=0), k=0, v=0) == 0
    assert _attend(lib, batch=_batch(rows=0), q=0, out=0, ws=0) == 0


def _attend(lib, cache=None, batch=None, q=A, qs=512, heads=4, scale=0.1, longest=1, mods=None, out=A, lse=0, ws=A, size=1 << 40):
    return lib.dsa_paged_attention(ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()), q, qs, heads, scale, longest,
                                   None if mods is None else ctypes.byref(mods), out, lse, ws, size, None)


@pytest.mark.parametrize("kw,status,word", BAD_CACHES)
def test_attention_rejects_bad_caches(lib, kw, status, word):
    _said(lib, _attend(lib, cache=_cache(**kw)), status, word)


@pytest.mark.parametrize("kw,status,word", BAD_BATCHES + [(dict(B=4097), UNSUPPORTED, "num_requests"),
                                                          (dict(stride=(1 << 24) + 1), UNSUPPORTED, "2^30"),
                                                          (dict(stride=1 << 24, B=4096, rows=4096), UNSUPPORTED, "2^31")])
def test_attention_rejects_bad_batches(lib, kw, status, word):
    _said(lib, _attend(lib, batch=_batch(**kw)), status, word)


@pytest.mark.parametrize("kw,status,word", [
    (dict(q=0), INVALID, "q is NULL"), (dict(q=A + 8), INVALID, "aligned"), (dict(qs=511), INVALID, "stride"),
    (dict(qs=504), INVALID, "stride"), (dict(heads=0), INVALID, "q_heads"), (dict(heads=3), INVALID, "multiple"),
    (dict(heads=130, qs=1 << 15), UNSUPPORTED, "per K/V head"), (dict(scale=0.0), INVALID, "scale"),
    (dict(scale=float("nan")), INVALID, "scale"), (dict(scale=float("inf")), INVALID, "scale"), (dict(scale=-1.0), INVALID, "scale"),
    (dict(longest=0), INVALID, "max_query_len"), (dict(out=0), INVALID, "out is NULL"), (dict(out=A + 4), INVALID, "aligned"),
    (dict(lse=A + 2), INVALID, "lse"), (dict(ws=0), WORKSPACE, "workspace"), (dict(size=64), WORKSPACE, "workspace"),
    (dict(ws=A + 16), INVALID, "aligned")])
def test_attention_rejects_bad_arguments(lib, kw, status, word):
    _said(lib, _attend(lib, **kw), status, word)


@pytest.mark.parametrize("cap,reserved,slopes,prefix,word", [(-1.0, 0, 0, 0, "softcap"), (float("nan"), 0, 0, 0, "softcap"),
                                                             (float("inf"), 0, 0, 0, "softcap"), (0.0, 1, 0, 0, "reserved"),
                                                             (0.0, 0, A + 2, 0, "aligned"), (0.0, 0, 0, A + 1, "aligned")])
def test_attention_rejects_bad_mods(lib, cap, reserved, slopes, prefix, word):
    from deepseek_sparse_mla_gb300._lib import DsaAttnMods
    _said(lib, _attend(lib, mods=DsaAttnMods(cap, reserved, slopes, prefix)), INVALID, word)


def test_attention_workspace_is_sized_by_heads_and_rows(lib):
    size = lib.dsa_paged_attention_workspace_bytes
    assert size(0, 1, 1) == 0 and size(8, 0, 1) == 0 and size(8, 3, 1) == 0 and size(8, 1, 0) == 0
    small, large = size(8, 1, 1), size(8, 1, 4096)
    assert 0 < small < large
    assert size(16, 2, 1) == small                          # heads per K/V head, not K/V heads
    assert _attend(lib, size=size(4, 2, 1) - 1) == WORKSPACE


def _plan(lib, lens=A, new=A, B=2, P=64, table=A, stride=8, free=A, cap=100, count=A, rows=4, out=A, qsl=A, slots=A, pos=A,
          count_out=A, ws=A, size=256):
    return lib.dsa_step_plan(lens, new, B, P, table, stride, free, cap, count, rows, out, qsl, slots, pos, count_out, ws, size, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(lens=0), INVALID, "NULL"), (dict(new=0), INVALID, "NULL"), (dict(table=0), INVALID, "NULL"), (dict(count=0), INVALID, "NULL"),
    (dict(out=0), INVALID, "NULL"), (dict(qsl=0), INVALID, "NULL"), (dict(count_out=0), INVALID, "NULL"),
    (dict(lens=A + 2), INVALID, "aligned"), (dict(slots=A + 4), INVALID, "aligned"), (dict(B=0), INVALID, "num_requests"),
    (dict(B=4097), UNSUPPORTED, "num_requests"), (dict(P=0), INVALID, "page_size"), (dict(P=24), INVALID, "page_size"),
    (dict(P=2048), INVALID, "page_size"), (dict(stride=0), INVALID, "stride"), (dict(cap=-1), INVALID, "negative"),
    (dict(rows=-1), INVALID, "negative"), (dict(size=64), WORKSPACE, "workspace"), (dict(ws=A + 4), INVALID, "aligned")])
def test_step_plan_rejects_bad_arguments(lib, kw, status, word):
    _said(lib, _plan(lib, **kw), status, word)


def _release(lib, done=A, lens=A, B=2, P=64, table=A, stride=8, pages=100, free=A, cap=100, count=A, ws=A, size=256):
    return lib.dsa_pages_release(done, lens, B, P, table, stride, pages, free, cap, count, ws, size, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(done=0), INVALID, "NULL"), (dict(lens=0), INVALID, "NULL"), (dict(table=0), INVALID, "NULL"), (dict(free=0), INVALID, "NULL"),
    (dict(count=0), INVALID, "NULL"), (dict(count=A + 2), INVALID, "aligned"), (dict(B=0), INVALID, "num_requests"),
    (dict(B=4097), UNSUPPORTED, "num_requests"), (dict(P=3), INVALID, "page_size"), (dict(stride=0), INVALID, "stride"),
    (dict(pages=0), INVALID, "num_pages"), (dict(size=64), WORKSPACE, "workspace")])
def test_release_rejects_bad_arguments(lib, kw, status, word):
    _said(lib, _release(lib, **kw), status, word)


def test_the_binding_rejects_tensors_that_do_not_fit():
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)   # noqa: E731
    with pytest.raises(ValueError, match="k_codes"):
        dsa.BlockKvCache.of(torch.zeros(4, 2, 64, 64, dtype=torch.uint8), *(None,) * 3)
    codes = torch.zeros(4, 2, 64, 128, dtype=torch.uint8)   # what lies on the host is refused
    with pytest.raises(ValueError, match="CUDA"):
        dsa.BlockKvCache.of(codes, codes.clone(), torch.ones(4, 2), torch.ones(4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        dsa.PagePool.of(i32(8), i32(1))
    with pytest.raises(ValueError, match="seq_lens"):
        dsa.step_plan(dsa.PagePool(8, device="cpu"), torch.zeros(2), i32(2), i32(2, 4), 64, 8)
