"""Refusals of the chunk attention and the page pool calls, checked before any launch (no GPU).

The raw C calls pass fake, never dereferenced device pointers: every case is turned down by the
argument checks, so no CUDA call is made."""

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


def _geom(H=8, Hk=2, D=128, dtype=0, cache=0):
    return B.KVGeometry(H, Hk, D, 0.0, dtype, cache)


def _cache(k=F, v=F + 0x1000, ps=16 * 2 * 128, rs=2 * 128, hs=128, page=16, pages=10, ksc=None,
           vsc=None):
    return B.KVCache(k, v, ps, rs, hs, page, pages, ksc, vsc)


def _chunk(geom=None, cache=None, **kw):
    a = dict(q=F, qs=1024, rows=5, kept=F, lens=F, rs=F, batch=3, table=F, W=8, window=0,
             out=F + 0x100000, lse=F, ws=F, wsb=1 << 40)
    a.update(kw)
    return B.lib().mla_chunk_attention(
        ctypes.byref(geom or _geom()), a["q"], a["qs"], a["rows"], ctypes.byref(cache or _cache()),
        a["kept"], a["lens"], a["rs"], a["batch"], a["table"], a["W"], a["window"], a["out"],
        a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(kept=None), dict(lens=None), dict(rs=None), dict(table=None),
    dict(out=None), dict(rows=-1), dict(batch=0), dict(batch=65536), dict(W=0), dict(W=2 ** 28),
    dict(window=-1), dict(qs=1000), dict(qs=1026), dict(q=F + 4), dict(table=F + 8),
    dict(rs=F + 4), dict(lse=F + 2), dict(ws=F + 16), dict(out=F), dict(out=F + 1024),
    dict(geom=_geom(H=7)), dict(geom=_geom(D=100)), dict(geom=_geom(D=264)),
    dict(geom=_geom(dtype=7)), dict(cache=_cache(k=None)), dict(cache=_cache(v=F + 8)),
    dict(cache=_cache(page=0)), dict(cache=_cache(rs=100)), dict(cache=_cache(ksc=F)),
])
def test_chunk_rejects(kw):
    assert _chunk(**kw) == B.MLA_ERR_INVALID_ARG
    assert B.mla_last_error() != ""


def test_chunk_unsupported_and_workspace():
    assert _chunk(_geom(cache=1)) == B.MLA_ERR_UNSUPPORTED
    assert _chunk(rows=2 ** 29, qs=1024) == B.MLA_ERR_UNSUPPORTED
    assert _chunk(ws=None) == B.MLA_ERR_WORKSPACE
    assert _chunk(wsb=256) == B.MLA_ERR_WORKSPACE
    assert _chunk(rows=0, q=None, out=None, ws=None, wsb=0) == B.MLA_OK      # no work
    small = B.mla_chunk_workspace_bytes(8, 2, 128, 3, 5, 16, 8)
    large = B.mla_chunk_workspace_bytes(8, 2, 128, 3, 5000, 16, 4096)
    assert 0 < small <= large
    assert B.mla_chunk_workspace_bytes(8, 2, 128, 3, 0, 16, 8) == 0
    with pytest.raises(B.MlaError):
        B.mla_chunk_workspace_bytes(8, 3, 128, 3, 5, 16, 8)
    n = ctypes.c_size_t(0)
    assert B.lib().mla_chunk_workspace_bytes(ctypes.byref(_geom()), 3, 5, 16, 8, None) == \
        B.MLA_ERR_INVALID_ARG
    assert B.lib().mla_chunk_workspace_bytes(None, 3, 5, 16, 8, ctypes.byref(n)) == \
        B.MLA_ERR_INVALID_ARG


def _fork(**kw):
    a = dict(src=F, lens=F + 0x1000, held=F + 0x2000, batch=4, table=F + 0x3000, W=8, page=16,
             pages=40, shares=F + 0x4000, free=F + 0x5000, cap=10, span=F + 0x6000,
             lens_out=F + 0x7000, held_out=F + 0x8000, shares_out=F + 0x9000,
             span_out=F + 0xA000, missing=F + 0xB000, msrc=F + 0xC000, mdst=F + 0xD000,
             mrows=F + 0xE000, moves=F + 0xF000)
    a.update(kw)
    return B.lib().mla_page_fork(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=65536), dict(W=0), dict(page=0), dict(pages=0), dict(cap=0),
    dict(W=2 ** 30), dict(pages=2 ** 30 + 1), dict(src=None), dict(table=None),
    dict(shares_out=None), dict(moves=None), dict(mrows=F + 8), dict(lens_out=F + 0x1000),
    dict(held_out=F + 0x2000), dict(span_out=F + 0x6000), dict(msrc=F + 0xD000),
    dict(table=F + 0x5000), dict(shares_out=F + 0x4010), dict(lens_out=F),
])
def test_page_fork_rejects(kw):
    assert _fork(**kw) == B.MLA_ERR_INVALID_ARG
    assert "page fork" in B.mla_last_error()


def _release(**kw):
    a = dict(kept=F, held=F + 0x1000, batch=4, table=F + 0x2000, W=8, page=16, pages=40,
             shares=F + 0x3000, free=F + 0x4000, cap=40, span=F + 0x5000, held_out=F + 0x6000,
             shares_out=F + 0x7000, span_out=F + 0x8000, released=F + 0x9000)
    a.update(kw)
    return B.lib().mla_page_release(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(W=0), dict(page=0), dict(pages=0), dict(cap=39), dict(W=2 ** 30),
    dict(kept=None), dict(free=None), dict(released=None), dict(span=F + 0x5008),
    dict(held_out=F + 0x1000), dict(free=F + 0x2000), dict(span_out=F + 0x5000),
    dict(shares_out=F + 0x2FF0), dict(held_out=F + 0x7000),
])
def test_page_release_rejects(kw):
    assert _release(**kw) == B.MLA_ERR_INVALID_ARG
    assert "page release" in B.mla_last_error()


def _compact(**kw):
    a = dict(held=F, batch=4, table=F + 0x1000, W=8, pages=40, shares=F + 0x2000,
             table_out=F + 0x3000, shares_out=F + 0x4000, free=F + 0x5000, cap=40,
             span=F + 0x6000, msrc=F + 0x7000, mdst=F + 0x8000, moves=F + 0x9000, ws=F + 0xA000,
             wsb=1 << 20)
    a.update(kw)
    return B.lib().mla_page_compact(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(W=0), dict(pages=0), dict(cap=39), dict(held=None), dict(table_out=None),
    dict(msrc=None), dict(moves=F + 0x9004), dict(ws=F + 0xA010), dict(table_out=F + 0x1010),
    dict(shares_out=F + 0x2010), dict(msrc=F + 0x8000), dict(free=F), dict(ws=F + 0x3000),
    dict(table_out=F + 0x2000),
])
def test_page_compact_rejects(kw):
    assert _compact(**kw) == B.MLA_ERR_INVALID_ARG
    assert B.mla_last_error() != ""


def test_page_compact_workspace_is_checked():
    assert _compact(ws=None) == B.MLA_ERR_WORKSPACE
    assert _compact(wsb=128) == B.MLA_ERR_WORKSPACE
    assert B.lib().mla_page_compact_workspace_bytes(0, F) == B.MLA_ERR_INVALID_ARG
    assert B.lib().mla_page_compact_workspace_bytes(5, None) == B.MLA_ERR_INVALID_ARG


def _copy(view=None, n=1, **kw):
    a = dict(page=16, pages=10, src=F + 0x1000, dst=F + 0x2000, rows=None, moves=None, cap=4)
    a.update(kw)
    v = dict(base=F, ps=16 * 256, rs=256, hs=128, heads=2, width=128)
    v.update(view or {})
    views = (B.PageView * max(1, n))(*[B.PageView(*v.values()) for _ in range(n)])
    return B.lib().mla_page_copy(views, n, *a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(n=129), dict(page=0), dict(pages=0), dict(cap=-1), dict(src=None),
    dict(dst=F + 8), dict(rows=F + 4), dict(moves=F + 4), dict(view=dict(base=None)),
    dict(view=dict(base=F + 8)), dict(view=dict(heads=0)), dict(view=dict(width=8)),
    dict(view=dict(width=120)), dict(view=dict(ps=-16)), dict(view=dict(rs=120)),
    dict(view=dict(hs=64)), dict(view=dict(rs=0)),
])
def test_page_copy_rejects(kw):
    assert _copy(**kw) == B.MLA_ERR_INVALID_ARG
    assert "page copy" in B.mla_last_error()


def test_page_copy_no_moves_and_large_pages():
    assert _copy(cap=0, src=None, dst=None) == B.MLA_OK
    assert B.lib().mla_page_copy(None, 1, 16, 10, F, F, None, None, 4, None) == \
        B.MLA_ERR_INVALID_ARG
    big = dict(width=2 ** 30, hs=2 ** 30, rs=2 ** 31, ps=2 ** 41, heads=2)
    assert _copy(view=big, page=2 ** 10) == B.MLA_ERR_UNSUPPORTED


# ------------------------------------------------------------------ the binding's own checks

def _t(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_checks_shapes_types_and_devices():
    q, kc = _t(5, 8, 64, dtype=torch.bfloat16), _t(4, 16, 2, 64, dtype=torch.bfloat16)
    a = dict(q=q, k_cache=kc, v_cache=kc, kept_lens=_t(3), cache_lens=_t(3), row_start=_t(4),
             page_table=_t(3, 2))
    for bad in (dict(row_start=_t(3)), dict(kept_lens=_t(4)), dict(cache_lens=_t(3).long()),
                dict(page_table=_t(3)), dict(q=q.float()), dict(k_cache=kc.half()),
                dict(v_cache=kc[:3]), dict(q=q.transpose(0, 1)),
                dict(out=_t(5, 8, 32, dtype=torch.bfloat16)), dict(lse=_t(5, 8))):
        with pytest.raises(ValueError):
            B.mla_chunk_attention(**{**a, **bad})
    with pytest.raises(ValueError, match="CUDA"):          # (all else is right)
        B.mla_chunk_attention(**a)
    f = dict(src_of=_t(3), cache_lens=_t(3), held_pages=_t(3), page_table=_t(3, 4),
             shares=_t(9), free_pages=_t(9), free_span=_t(2), page_size=8)
    for bad in (dict(src_of=_t(2)), dict(free_span=_t(3)), dict(shares=_t(9).long()),
                dict(page_table=_t(3)), dict(held_pages=_t(6)[::2])):
        with pytest.raises(ValueError):
            B.mla_page_fork(**{**f, **bad})
    with pytest.raises(ValueError):
        B.mla_page_release(_t(3), _t(3), _t(3, 4), _t(9), _t(9), _t(2), 8, out=(_t(3), _t(9)))
    with pytest.raises(ValueError):
        B.mla_page_compact(_t(3), _t(3, 4), _t(9), _t(9, 1))
    for caches in ([], [_t(4, 16)], [kc, kc[:3]], [kc, _t(4, 8, 2, 64)], [kc.transpose(2, 3)],
                   [_t(0, 16, 64)]):
        with pytest.raises(ValueError):
            B.mla_page_copy(caches, _t(2), _t(2))
    with pytest.raises(ValueError):
        B.mla_page_copy([kc], _t(2), _t(3))
    with pytest.raises(ValueError, match="CUDA"):
        B.mla_page_copy([kc], _t(2), _t(2))


def test_package_exports_the_calls():
    import mla_attention_speculative_gb300 as mla
    for name in ("mla_chunk_attention", "mla_page_fork", "mla_page_release", "mla_page_compact",
                 "mla_page_copy", "PreparedChunkAttention", "PreparedPageFork",
                 "PreparedPageRelease", "PreparedPageCompact", "PreparedPageCopy"):
        assert getattr(mla, name) is getattr(B, name)
