"""Forks that meet page ids outside the pool: in the free list, in a source's whole pages, in its
last one.  The call reports them and mla_page_copy passes over the moves."""

import numpy as np
import pytest
import torch

from oracle import page_pool as O
from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib
from test_page_pool_gpu import DEV, check_fork, i32, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    B.lib()
    yield
    torch.cuda.synchronize()
    B.mla_device_status()


# table row 0 holds three pages of four rows; slots 1 and 2 take them
@pytest.mark.parametrize("row,lens,free,bad", [
    ([3, 1, 2], 10, [4, 5], False),
    ([3, 1, 2], 10, [4, 6], True),          # the second slot's page
    ([3, 1, 2], 10, [-1, 5], True),
    ([3, 1, 6], 10, [4, 5], True),          # the source's last page
    ([3, 1, -2], 10, [4, 5], True),
    ([3, 1, -2], 8, [9, 9], False),         # no rows in it, and none taken
    ([3, 7, 2], 10, [4, 5], True),          # a whole one
    ([3, 1, 6], 10, [4], True),
    ([3, 1, 6], 10, [], False),             # the list has run out: nothing is read
])
def test_fork_reports_bad_ids(row, lens, free, bad):
    table = np.full((3, 4), -1)
    table[0, :3] = row
    args = ([-1, 0, 0], [lens, 0, 0], [3, 0, 0], table, [0] * 6, free + [-1], [0, len(free)], 4)
    assert O.page_fork(*args)[7] == bad
    got, moves = check_fork(*args)
    cache = torch.arange(6 * 4 * 16, device=DEV, dtype=torch.float32).view(6, 4, 16)
    want = O.page_copy(cache.cpu().numpy(), moves, 4)
    B.mla_page_copy([cache], got.move_src, got.move_dst, got.moves, got.move_rows)
    outside = any(not 0 <= m < 6 for x in moves for m in x[:2])
    assert status() == outside and np.array_equal(cache.cpu().numpy(), want)
