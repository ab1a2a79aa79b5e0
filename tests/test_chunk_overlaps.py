"""The chunk attention refuses outputs and workspaces that overlap another buffer of the call, before
any launch (no GPU: the pointers are fake and never dereferenced)."""

import ctypes

import pytest
import torch

from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib

# 5 rows of 8 heads on 2 of 128, 3 sequences of 8 pages, each buffer a megabyte or more apart
H, HK, D, ROWS, BATCH, W = 8, 2, 128, 5, 3, 8
AT = {name: (i + 1) << 24 for i, name in enumerate(
    ("q", "out", "lse", "ws", "kept", "lens", "row_start", "table", "k", "v", "k_scale",
     "v_scale"))}
SIZE = dict(q=ROWS * H * D * 2, out=ROWS * H * D * 2, lse=ROWS * H * 4, kept=BATCH * 4,
            lens=BATCH * 4, row_start=(BATCH + 1) * 4, table=BATCH * W * 4, k_scale=HK * 4,
            v_scale=HK * 4)


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    SIZE["ws"] = B.mla_chunk_workspace_bytes(H, HK, D, BATCH, ROWS, 64, W,
                                             cache_dtype=torch.float8_e4m3fn)
    yield


def call(**kw):
    a = {**AT, **kw}
    geom = B.KVGeometry(H, HK, D, 0.0, 0, 2)
    cache = B.KVCache(a["k"], a["v"], 64 * HK * D, HK * D, D, 64, 10, a["k_scale"], a["v_scale"])
    return B.lib().mla_chunk_attention(
        ctypes.byref(geom), a["q"], H * D, ROWS, ctypes.byref(cache), a["kept"], a["lens"],
        a["row_start"], BATCH, a["table"], W, 0, a["out"], a["lse"], a["ws"], SIZE["ws"], None)


PAIRS = [(a, b) for a in ("out", "lse", "ws") for b in SIZE if a != b] + [
    (a, "ws") for a in ("out", "lse")]


@pytest.mark.parametrize("written,other", PAIRS)
def test_chunk_refuses_overlaps(written, other):
    step = 256 if written == "ws" else 16
    first, last = AT[other], AT[other] + (SIZE[other] - 1) // step * step
    # at the same place, in the other's last bytes, with its own last ones in the other's first
    for at in (first, last, first - (SIZE[written] - 1) // step * step):
        assert call(**{written: at}) == B.MLA_ERR_INVALID_ARG
        assert "overlaps" in B.mla_last_error()
