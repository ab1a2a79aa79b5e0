"""Refusals of the paged-step entry points at the largest sizes (no GPU): like
the other refusals they are turned down before any CUDA call is made, so the
device pointers are fake and never dereferenced."""

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


def test_append_latent_counts_the_largest_rows():
    # 2^31 - 1 rows of four heads take more thread blocks than a grid has
    geom = B.make_geometry(H=4, r=512, n=128, v=128, rope=64, dtype=torch.bfloat16)
    st = B.lib().mla_append_latent(
        ctypes.byref(geom), F, 4 * 192, F, 576, F, ctypes.c_float(1e-6), F, 100, 1, F, F,
        2 ** 31 - 1, F, F, F, F, 512, 64, 100, None)
    assert st == B.MLA_ERR_UNSUPPORTED
    assert "too many" in B.mla_last_error()


@pytest.mark.parametrize("at,value", [(8, 2 ** 32 + 5), (8, 2 ** 31), (7, -2 ** 31 - 1)])
def test_numbers_beyond_32_bits_are_refused(at, value):
    # (a window of 2^32 + 5 is not one of 5)
    args = [F, F, 64, F, F, 3, F, 8, 0, F, F, F, 0]
    args[at] = value
    with pytest.raises(ValueError, match="32-bit"):
        B._PreparedCall()._prepare("mla_decode_attention", args, torch.device("cuda", 0), ())


def test_the_package_exports_the_paged_steps():
    import mla_attention_speculative_gb300 as mla
    for name in ("mla_page_step", "mla_append_latent", "mla_append_kv", "mla_decode_attention",
                 "mla_decode_workspace_bytes", "PageStep", "PreparedPageStep",
                 "PreparedAppendLatent", "PreparedAppendKV", "PreparedDecodeAttention"):
        assert name in mla.__all__ and getattr(mla, name) is getattr(B, name)


def _decode(**kw):
    geom = B.KVGeometry(8, 2, 128, 0.0, 0, 0)
    cache = B.KVCache(F, F + 0x1000, 16 * 2 * 128, 2 * 128, 128, 16, 10, None, None)
    a = dict(q=F, qs=1024, lens=F, batch=3, table=F, W=4096, window=0, out=F + 0x100000, lse=F,
             ws=F, wsb=0)
    a.update(kw)
    v = list(a.values())
    return B.lib().mla_decode_attention(ctypes.byref(geom), v[0], v[1], ctypes.byref(cache),
                                        *v[2:], None)


@pytest.mark.parametrize("kw", [dict(out=F + 16), dict(out=F - 16), dict(out=F, qs=1032),
                                dict(out=F + 2 * 1032 * 2 + 2032, qs=1032),
                                dict(q=F + 3 * 2048 - 16, out=F)])
def test_decode_out_may_be_q_but_not_overlap_it(kw):
    assert _decode(**kw) == B.MLA_ERR_INVALID_ARG
    assert "overlaps q" in B.mla_last_error()


@pytest.mark.parametrize("kw", [dict(), dict(out=F), dict(out=F + 3 * 2048), dict(out=F - 3 * 2048),
                                dict(out=F + (2 * 1032 + 1024) * 2, qs=1032)])
def test_decode_out_beside_q_passes(kw):
    # (the workspace is what is refused here)
    assert _decode(**kw) == B.MLA_ERR_WORKSPACE
