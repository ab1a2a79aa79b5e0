"""The softmax scales that the paged attentions' binding takes (no GPU): the library holds them in
fp32, where 0 asks for 1/sqrt(head_dim), so one that rounds to 0 must not get there."""

import math

import pytest
import torch

from mla_attention_speculative_gb300 import binding as B

KV = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
I32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731


def calls(scale):
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    yield lambda: B.mla_chunk_attention(q, KV, KV, I32(3), I32(3), I32(4), I32(3, 2), scale=scale)
    yield lambda: B.mla_decode_attention(q, KV, KV, I32(3), I32(3, 2), scale=scale)


@pytest.mark.parametrize("scale", [0.0, -1.0, 1e-46, 5e-324, 1e39, math.inf, math.nan])
def test_scales_that_fp32_does_not_hold_are_refused(scale):
    for f in calls(scale):
        with pytest.raises(ValueError, match="scale"):
            f()


@pytest.mark.parametrize("scale", [None, 1e-45, 0.125, torch.tensor(2.0), 1])
def test_scales_that_it_holds_are_taken(scale):
    for f in calls(scale):
        with pytest.raises(ValueError, match="CUDA"):      # (all else is right)
            f()
