"""What the chunk attention writes to its workspace, with the shares found inside the kernel (up to
256 sequences) or by a launch ahead of it, with units that may be cut and with tables too short for
that: the bytes asked for and no others, whatever they held."""

import pytest
import torch

from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib
from test_chunk_gpu import BF16, DEV, E4M3, FP32, case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    B.lib()
    yield
    torch.cuda.synchronize()
    B.mla_device_status()


@pytest.mark.parametrize("dtype,cache,D", [(BF16, BF16, 64), (BF16, BF16, 256), (BF16, E4M3, 128),
                                           (FP32, FP32, 64)])
@pytest.mark.parametrize("batch,kept", [(3, 40), (3, 900), (300, 40), (300, 900), (2500, 20),
                                        (2500, 600)])
def test_chunk_writes_its_workspace_alone(dtype, cache, D, batch, kept):
    kept = [(kept + 7 * b) % (kept + 1) for b in range(batch)]
    new = [(3 * b) % 5 for b in range(batch)]
    c = case(kept, new, 2, 1, D, 16, dtype, cache, seed=batch + D)
    N, H, _ = c["q"].shape
    need = B.mla_chunk_workspace_bytes(H, 1, D, batch, N, 16, c["page_table"].shape[1], dtype,
                                       cache)
    for fill in (0x00, 0x7F, 0xFF):
        guarded = torch.full((need + (64 << 20),), 0x5A, dtype=torch.uint8, device=DEV)
        guarded[:need] = fill
        out = torch.full(c["q"].shape, 7.0, dtype=dtype, device=DEV)
        lse = torch.full((N, H), 7.0, device=DEV)
        B.mla_chunk_attention(**c, out=out, lse=lse, workspace=guarded[:need])
        torch.cuda.synchronize()
        assert (guarded[need:] == 0x5A).all()
        if fill:
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        first = out, lse
    check(c, *first)
