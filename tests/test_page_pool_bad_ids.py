"""Pin of the oracle's fork: page ids outside the pool are noticed wherever a slot takes one."""

import pytest

from oracle import page_pool as O


@pytest.mark.parametrize("row,free,bad", [
    ([3, 1, 2], [4], False), ([3, 1, 2], [6], True), ([3, 1, 2], [-1], True),
    ([3, 1, 6], [4], True), ([3, -1, 2], [4], True), ([3, 1, 6], [], False),
])
def test_fork_notices_bad_ids(row, free, bad):
    out = O.page_fork([-1, 0], [10, 0], [3, 0], [row, [-1] * 3], [0] * 6, free, [0, len(free)], 4)
    assert out[7] == bad
    assert out[6] == ([(row[2], free[0], 2)] if free else [])
