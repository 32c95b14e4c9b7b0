"""The 4-bit cache's append and attention and the rotating appends reject bad arguments on the host, before any launch (no GPU)."""
import ctypes

import pytest

from test_dense_refusals import A, BAD_BATCHES, INVALID, UNSUPPORTED, WORKSPACE, _batch, _said
from test_dense_refusals import _cache as _cache8


def _cache(**kw):
    from deepseek_sparse_mla_gb300._lib import DsaKv4Cache
    f = dict(k=A, v=A, ks=A, vs=A, pages=16, P=64, heads=2, reserved=0)
    f.update(kw)
    return DsaKv4Cache(f["k"], f["v"], f["ks"], f["vs"], f["pages"], f["P"], f["heads"], f["reserved"])


def _rope(**kw):
    from deepseek_sparse_mla_gb300._lib import DsaRope
    f = dict(cs=A, positions=300, dim=64, interleaved=0, heads=16, q=A, qs=2048, out=A, os=2048)
    f.update(kw)
    return DsaRope(f["cs"], f["positions"], f["dim"], f["interleaved"], f["heads"], f["q"], f["qs"], f["out"], f["os"])


BAD_CACHES = [(dict(k=0), INVALID, "NULL"), (dict(ks=0), INVALID, "NULL"), (dict(vs=0), INVALID, "NULL"), (dict(k=A + 16), INVALID, "32-byte"),
              (dict(v=A + 8), INVALID, "32-byte"), (dict(ks=A + 8), INVALID, "16-byte"), (dict(vs=A + 2), INVALID, "16-byte"),
              (dict(pages=0), INVALID, "num_pages"), (dict(P=48), UNSUPPORTED, "page_size"), (dict(P=256), UNSUPPORTED, "page_size"),
              (dict(P=8), UNSUPPORTED, "page_size"), (dict(heads=0), INVALID, "kv_heads"), (dict(pages=1 << 30), UNSUPPORTED, "2^31"),
              (dict(reserved=1), INVALID, "reserved")]


def _append4(lib, cache=None, batch=None, k=A, ks=256, v=A, vs=256, rope=None):
    return lib.dsa_kv4_append(ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()), k, ks, v, vs,
                              None if rope is None else ctypes.byref(rope), None)


def _append8(lib, cache=None, batch=None, k=A, ks=256, v=A, vs=256, rope=None):
    return lib.dsa_kv8_append_rope(ctypes.byref(cache or _cache8()), ctypes.byref(batch or _batch()), k, ks, v, vs,
                                   None if rope is None else ctypes.byref(rope), None)


def _attend(lib, cache=None, batch=None, q=A, qs=512, heads=4, scale=0.1, longest=1, mods=None, out=A, lse=0, ws=A, size=1 << 40):
    return lib.dsa_kv4_attention(ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()), q, qs, heads, scale, longest,
                                 None if mods is None else ctypes.byref(mods), out, lse, ws, size, None)


APPENDS = pytest.mark.parametrize("append", [_append4, _append8], ids=["4", "8"])


@pytest.mark.parametrize("kw,status,word", BAD_CACHES)
def test_bad_caches(lib, kw, status, word):
    _said(lib, _append4(lib, cache=_cache(**kw)), status, word)
    _said(lib, _append4(lib, cache=_cache(**kw), rope=_rope()), status, word)
    _said(lib, _attend(lib, cache=_cache(**kw)), status, word)


@APPENDS
@pytest.mark.parametrize("kw,status,word", BAD_BATCHES)
def test_appends_reject_bad_batches(lib, append, kw, status, word):
    _said(lib, append(lib, batch=_batch(**kw), rope=_rope()), status, word)


@pytest.mark.parametrize("kw,status,word", BAD_BATCHES + [(dict(B=4097), UNSUPPORTED, "num_requests"),
                                                          (dict(stride=(1 << 24) + 1), UNSUPPORTED, "2^30"),
                                                          (dict(stride=1 << 24, B=4096, rows=4096), UNSUPPORTED, "2^31")])
def test_attention_rejects_bad_batches(lib, kw, status, word):
    _said(lib, _attend(lib, batch=_batch(**kw)), status, word)


@APPENDS
@pytest.mark.parametrize("kw,word", [(dict(k=0), "k is NULL"), (dict(v=0), "v is NULL"), (dict(k=A + 2), "aligned"), (dict(v=A + 8), "aligned"),
                                     (dict(ks=255), "stride"), (dict(vs=128), "stride"), (dict(vs=260), "stride")])
def test_appends_reject_bad_rows(lib, append, kw, word):
    _said(lib, append(lib, rope=_rope(), **kw), INVALID, word)
    if append is _append4:
        _said(lib, append(lib, **kw), INVALID, word)


@APPENDS
@pytest.mark.parametrize("kw,status,word", [
    (dict(cs=0), INVALID, "cos_sin is NULL"), (dict(cs=A + 8), INVALID, "aligned"), (dict(dim=0), UNSUPPORTED, "dim"),
    (dict(dim=48), UNSUPPORTED, "dim"), (dict(dim=160), UNSUPPORTED, "dim"), (dict(dim=-32), UNSUPPORTED, "dim"),
    (dict(interleaved=2), INVALID, "interleaved"), (dict(positions=299), INVALID, "positions"), (dict(positions=0), INVALID, "positions"),
    (dict(heads=-1), INVALID, "q_heads"), (dict(heads=0), INVALID, "without"), (dict(heads=0, q=0), INVALID, "without"),
    (dict(heads=65536, qs=1 << 24, os=1 << 24), UNSUPPORTED, "q_heads"), (dict(q=0), INVALID, "q is NULL"), (dict(out=0), INVALID, "q_out is NULL"),
    (dict(q=A + 8), INVALID, "aligned"), (dict(out=A + 2), INVALID, "aligned"), (dict(qs=2047), INVALID, "stride"),
    (dict(qs=2052), INVALID, "stride"), (dict(os=1920), INVALID, "stride"), (dict(os=4096), INVALID, "another stride")])
def test_appends_reject_bad_rotations(lib, append, kw, status, word):
    _said(lib, append(lib, rope=_rope(**kw)), status, word)


@APPENDS
def test_appends_reject_more_rows_and_heads_than_a_grid_holds(lib, append):
    rope = _rope(heads=65535, qs=1 << 23, os=1 << 23)
    _said(lib, append(lib, batch=_batch(B=1, rows=1 << 30), rope=rope), UNSUPPORTED, "too large")


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


def test_null_structs_and_calls_without_rows(lib):
    b, c = _batch(), _cache()
    _said(lib, lib.dsa_kv4_append(None, ctypes.byref(b), A, 256, A, 256, None, None), INVALID, "cache is NULL")
    _said(lib, lib.dsa_kv4_append(ctypes.byref(c), None, A, 256, A, 256, None, None), INVALID, "batch is NULL")
    _said(lib, _append8(lib), INVALID, "rope is NULL")
    _said(lib, lib.dsa_kv8_append_rope(None, ctypes.byref(b), A, 256, A, 256, ctypes.byref(_rope()), None), INVALID, "cache is NULL")
    _said(lib, lib.dsa_kv4_attention(None, ctypes.byref(b), A, 512, 4, 1.0, 1, None, A, None, A, 1 << 30, None), INVALID, "cache")
    _said(lib, lib.dsa_kv4_attention(ctypes.byref(c), None, A, 512, 4, 1.0, 1, None, A, None, A, 1 << 30, None), INVALID, "batch")
    none = _batch(rows=0)
    for append in (_append4, _append8):
        assert append(lib, batch=none, k=0, v=0, rope=_rope(q=0, out=0)) == 0
        _said(lib, append(lib, batch=none, k=0, v=0, rope=_rope(dim=48)), UNSUPPORTED, "dim")
    assert _append4(lib, batch=none, k=0, v=0) == 0 and _attend(lib, batch=none, q=0, out=0, ws=0) == 0


def test_a_cache_of_the_other_kind_is_refused(lib):
    b = ctypes.byref(_batch())
    with pytest.raises(ctypes.ArgumentError):
        lib.dsa_kv8_append(ctypes.byref(_cache()), b, A, 256, A, 256, None)
    with pytest.raises(ctypes.ArgumentError):
        lib.dsa_paged_attention(ctypes.byref(_cache()), b, A, 512, 4, 0.1, 1, None, A, 0, A, 1 << 40, None)
    with pytest.raises(ctypes.ArgumentError):
        lib.dsa_kv4_append(ctypes.byref(_cache8()), b, A, 256, A, 256, None, None)
    with pytest.raises(ctypes.ArgumentError):
        lib.dsa_kv4_attention(ctypes.byref(_cache8()), b, A, 512, 4, 0.1, 1, None, A, 0, A, 1 << 40, None)


def test_attention_workspace_is_that_of_the_8_bit_cache(lib):
    size = lib.dsa_paged_attention_workspace_bytes
    for longest in (1, 40):
        assert _attend(lib, batch=_batch(rows=64), longest=longest, size=size(4, 2, longest) - 1) == WORKSPACE


def test_the_binding_rejects_tensors_that_do_not_fit():
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    codes, exps = torch.zeros(4, 2, 64, 64, dtype=torch.uint8), torch.zeros(4, 2, 64, 4, dtype=torch.uint8)
    scales = torch.ones(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_codes"):
        dsa.Kv4Cache.of(torch.zeros(4, 2, 64, 128, dtype=torch.uint8), codes, exps, scales)
    with pytest.raises(ValueError, match="CUDA"):            # what lies on the host is refused
        dsa.Kv4Cache.of(codes, codes.clone(), exps, scales)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.RotaryTable.of(torch.zeros(10, 64))
    with pytest.raises(ValueError):
        dsa.RotaryTable.of(torch.zeros(10, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        dsa.RotaryTable.of(torch.zeros(640))
