"""Refusals of the paged-step entry points, checked before any launch (no GPU).

The raw C calls pass fake, never dereferenced device pointers: every case is
turned down by the argument checks, so no CUDA call is made."""

import ctypes

import pytest
import torch

from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib

F = 0x100000


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    yield


def _page_step(**kw):
    a = dict(kept=F, new=F + 0x1000, held=F + 0x2000, batch=4, table=F + 0x3000, W=8, page=16,
             pages=40, free=F + 0x4000, cap=10, span=F + 0x5000, lens=F + 0x6000,
             held_out=F + 0x7000, rs=F + 0x8000, pos=F + 0x9000, slots=F + 0xA000, rows=64,
             span_out=F + 0xB000, missing=F + 0xC000)
    a.update(kw)
    return B.lib().mla_page_step(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=65536), dict(W=0), dict(page=0), dict(pages=0), dict(cap=-1),
    dict(rows=-1), dict(W=2 ** 30), dict(kept=None), dict(table=None), dict(free=None),
    dict(span=None), dict(slots=None), dict(missing=None), dict(slots=F + 0xA008),
    dict(lens=F), dict(held_out=F + 0x2000), dict(span_out=F + 0x5000), dict(pos=F + 0x3010),
    dict(rs=F + 0x6000), dict(slots=F + 0x9000),
])
def test_page_step_rejects(kw):
    assert _page_step(**kw) == B.MLA_ERR_INVALID_ARG
    assert "page step" in B.mla_last_error()


def _geom(**kw):
    a = dict(H=4, r=512, n=128, v=128, rope=64, dtype=torch.bfloat16)
    a.update(kw)
    return B.make_geometry(**a)


def _latent(geom=None, **kw):
    a = dict(q=F, qs=4 * 192, kv=F, kvs=576, w=F, eps=1e-6, cs=F, table=100, inter=1, pos=F,
             slots=F, rows=3, qn=F, qr=F, c=F, k=F, cstr=512, kstr=64, cache=100)
    a.update(kw)
    a["eps"] = ctypes.c_float(a["eps"])
    return B.lib().mla_append_latent(ctypes.byref(geom or _geom()), *a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(geom=_geom(rope=24)), dict(geom=_geom(rope=0)), dict(geom=_geom(H=0)),
    dict(geom=_geom(r=2048)), dict(rows=-1), dict(table=0), dict(cache=0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(kv=None), dict(cs=None), dict(pos=None), dict(slots=None),
    dict(qn=None), dict(qr=None), dict(c=None), dict(k=None), dict(q=F + 2), dict(kvs=575),
    dict(kvs=577), dict(qs=100), dict(cstr=500), dict(kstr=32), dict(w=F + 8),
])
def test_append_latent_rejects(kw):
    assert _latent(**kw) == B.MLA_ERR_INVALID_ARG
    assert B.mla_last_error() != ""


def test_no_rows_is_no_work():
    assert _latent(rows=0) == B.MLA_OK
    assert _kv(rows=0) == B.MLA_OK


def _kv_geom(H=8, Hk=2, D=128, dtype=0, cache=0):
    return B.KVGeometry(H, Hk, D, 0.0, dtype, cache)


def _cache(k=F, v=F + 0x1000, ps=16 * 2 * 128, rs=2 * 128, hs=128, page=16, pages=10, ksc=None,
           vsc=None):
    return B.KVCache(k, v, ps, rs, hs, page, pages, ksc, vsc)


def _kv(geom=None, cache=None, **kw):
    a = dict(q=F, qs=1024, k=F, ks=256, v=F, vs=256, cs=F, table=100, rope=128, inter=0, pos=F,
             slots=F, rows=3, out=F + 0x100000)
    a.update(kw)
    return B.lib().mla_append_kv(ctypes.byref(geom or _kv_geom()), *a.values(),
                                 ctypes.byref(cache or _cache()), None)


BAD_GEOMS = [
    (dict(H=0), B.MLA_ERR_INVALID_ARG), (dict(H=7), B.MLA_ERR_INVALID_ARG),
    (dict(Hk=0), B.MLA_ERR_INVALID_ARG), (dict(D=0), B.MLA_ERR_INVALID_ARG),
    (dict(D=100), B.MLA_ERR_INVALID_ARG), (dict(D=264), B.MLA_ERR_INVALID_ARG),
    (dict(D=120, cache=2), B.MLA_ERR_INVALID_ARG), (dict(dtype=7), B.MLA_ERR_INVALID_ARG),
    (dict(dtype=2, cache=2), B.MLA_ERR_INVALID_ARG), (dict(cache=1), B.MLA_ERR_UNSUPPORTED),
    (dict(dtype=1, cache=2), B.MLA_ERR_UNSUPPORTED), (dict(H=131072), B.MLA_ERR_INVALID_ARG),
]
BAD_CACHES = [dict(k=None), dict(v=None), dict(k=F + 8), dict(page=0), dict(pages=0),
              dict(ps=-16), dict(rs=100), dict(hs=64), dict(ps=4), dict(ksc=F), dict(vsc=F)]


@pytest.mark.parametrize("kw,status", BAD_GEOMS)
def test_kv_geometry_is_checked(kw, status):
    assert _kv(_kv_geom(**kw)) == status
    assert _decode(_kv_geom(**kw)) == status


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_kv_cache_is_checked(kw):
    assert _kv(cache=_cache(**kw)) == B.MLA_ERR_INVALID_ARG
    assert _decode(cache=_cache(**kw)) == B.MLA_ERR_INVALID_ARG
    e4m3 = _kv_geom(cache=2)
    assert _kv(e4m3, cache=_cache(ksc=F + 2)) == B.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rope=-16), dict(rope=24), dict(rope=144), dict(table=0), dict(k=None),
    dict(v=None), dict(cs=None), dict(pos=None), dict(slots=None), dict(out=None),
    dict(q=F + 2), dict(qs=1000), dict(ks=128), dict(vs=260), dict(out=F + 16),
    dict(out=F, qs=1032),
])
def test_append_kv_rejects(kw):
    assert _kv(**kw) == B.MLA_ERR_INVALID_ARG
    assert B.mla_last_error() != ""


def _decode(geom=None, cache=None, **kw):
    a = dict(q=F, qs=1024, lens=F, batch=3, table=F, W=8, window=0, out=F, lse=F, ws=F, wsb=1 << 40)
    a.update(kw)
    return B.lib().mla_decode_attention(
        ctypes.byref(geom or _kv_geom()), a["q"], a["qs"], ctypes.byref(cache or _cache()),
        a["lens"], a["batch"], a["table"], a["W"], a["window"], a["out"], a["lse"], a["ws"],
        a["wsb"], None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(lens=None), dict(table=None), dict(out=None), dict(batch=0),
    dict(batch=65536), dict(W=0), dict(W=2 ** 28), dict(window=-1), dict(qs=1000), dict(qs=512),
    dict(q=F + 4), dict(table=F + 8), dict(lse=F + 2), dict(ws=F + 16),
])
def test_decode_rejects(kw):
    assert _decode(**kw) == B.MLA_ERR_INVALID_ARG
    assert B.mla_last_error() != ""


def test_decode_workspace_is_checked():
    need = B.mla_decode_workspace_bytes(8, 2, 128, 3, 16, 4096)
    if need:
        assert _decode(W=4096, ws=None, wsb=0) == B.MLA_ERR_WORKSPACE
        assert _decode(W=4096, wsb=need - 1) == B.MLA_ERR_WORKSPACE
    with pytest.raises(B.MlaError):
        B.mla_decode_workspace_bytes(8, 3, 128, 3, 16, 4096)
    out = ctypes.c_size_t(0)
    assert B.lib().mla_decode_workspace_bytes(ctypes.byref(_kv_geom()), 3, 16, 4,
                                              None) == B.MLA_ERR_INVALID_ARG
    assert B.lib().mla_decode_workspace_bytes(ctypes.byref(_kv_geom()), 3, 0, 4,
                                              ctypes.byref(out)) == B.MLA_ERR_INVALID_ARG


# ------------------------------------------------------------------ the binding's own checks

def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _append_kv_args(**kw):
    a = dict(q=_z(3, 8, 128), k=_z(3, 2, 128), v=_z(3, 2, 128), cos_sin=_z(9, 128, dtype=torch.float32),
             positions=_i(3), slots=torch.zeros(3, dtype=torch.int64), k_cache=_z(4, 16, 2, 128),
             v_cache=_z(4, 16, 2, 128))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,match", [
    (dict(), "CUDA device"),
    (dict(k=_z(3, 2, 128, dtype=torch.float16), v=_z(3, 2, 128, dtype=torch.float16)), "bf16 or fp32"),
    (dict(v=_z(3, 2, 64)), r"v must be \[3, 2, 128\]"),
    (dict(q=_z(2, 8, 128)), "q must be"),
    (dict(q=_z(3, 128, 8).transpose(1, 2)), "heads of a row"),
    (dict(positions=torch.zeros(3, dtype=torch.int64)), "positions must be torch.int32"),
    (dict(slots=_i(3)), "slots must be torch.int64"),
    (dict(k_cache=_z(4, 16, 4, 128)), "k_cache must be"),
    (dict(v_cache=_z(4, 2, 16, 128).transpose(1, 2)), "same strides"),
    (dict(k_cache=_z(4, 16, 2, 128, dtype=torch.float16),
          v_cache=_z(4, 16, 2, 128, dtype=torch.float16)), "cache must be"),
    (dict(k_scale=_z(2)), "k_scale must be torch.float32"),
    (dict(cos_sin=_z(9, 128)), "cos_sin must be"),
    (dict(q=None, q_out=_z(3, 8, 128)), "needs q"),
])
def test_append_kv_binding_rejects(kw, match):
    with pytest.raises(ValueError, match=match):
        B.mla_append_kv(**_append_kv_args(**kw))


@pytest.mark.parametrize("kw,match", [
    (dict(), "CUDA device"),
    (dict(cache_lens=torch.zeros(2, dtype=torch.int64)), "cache_lens must be torch.int32"),
    (dict(page_table=_i(3, 4)), "page_table must be"),
    (dict(out=_z(2, 8, 64)), "out must be"),
    (dict(lse=_z(2, 8)), "lse must be torch.float32"),
    (dict(q=_z(2, 8, 64)), "k_cache must be"),
    (dict(scale=0.0), "CUDA device|scale must be positive"),
])
def test_decode_binding_rejects(kw, match):
    a = dict(q=_z(2, 8, 128), k_cache=_z(4, 16, 2, 128), v_cache=_z(4, 16, 2, 128),
             cache_lens=_i(2), page_table=_i(2, 4))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        B.mla_decode_attention(**a)


@pytest.mark.parametrize("kw,match", [
    (dict(), "CUDA device"),
    (dict(kv=_z(3, 576, dtype=torch.float16)), "bf16 or fp32"),
    (dict(c_kv=_z(4, 16, 256)), "c_kv must be"),
    (dict(k_rope=_z(5, 16, 64)), "same rows"),
    (dict(norm_weight=_z(512, dtype=torch.float32)), "norm_weight must be"),
    (dict(q=_z(2, 4, 192)), "with kv's rows"),
    (dict(q_nope=_z(3, 4, 64)), "q_nope must be"),
])
def test_append_latent_binding_rejects(kw, match):
    a = dict(q=_z(3, 4, 192), kv=_z(3, 576), cos_sin=_z(9, 64, dtype=torch.float32),
             positions=_i(3), slots=torch.zeros(3, dtype=torch.int64), c_kv=_z(4, 16, 512),
             k_rope=_z(4, 16, 64))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        B.mla_append_latent(**a)


@pytest.mark.parametrize("kw,match", [
    (dict(), "CUDA device"), (dict(kept_lens=_i(3)), "kept_lens must be"),
    (dict(free_span=_i(3)), "free_span must be"), (dict(max_rows=-1), "max_rows"),
    (dict(page_table=_i(4, 8).t()), "kept_lens must be|contiguous"),
])
def test_page_step_binding_rejects(kw, match):
    a = dict(kept_lens=_i(4), new_tokens=_i(4), held_pages=_i(4), page_table=_i(4, 8),
             free_pages=_i(9), free_span=_i(2), page_size=16, num_pages=40, max_rows=12)
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        B.mla_page_step(**a)
