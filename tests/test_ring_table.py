"""The page table of a window that moves over a rollout (no GPU): the rows that a chunk sees lie in pages of
their own, whatever the sizes."""
import itertools

import numpy as np
import pytest

from kv_cache_tempcache_gb300.layer import ring_table
from oracle import paged_oracle as P


@pytest.mark.parametrize("page,sinks,window,chunk", list(itertools.product((16, 32), (0, 1, 16, 33), (1, 16, 50), (1, 7, 40))))
@pytest.mark.parametrize("block", [0, 1, 3])
def test_rows_that_are_seen_share_no_slot(page, sinks, window, chunk, block):
    rows = 20 * page + 5
    table, pages = ring_table(rows, page, sinks, window, chunk)
    table = table.numpy()
    assert len(table) == 21 and table.min() >= 0 and table.max() == pages - 1
    keep = -(-sinks // page)
    assert pages <= keep + (window + chunk) // page + 2
    holds = np.full(pages * page, -1)                         # the row that each slot holds
    for at in range(0, rows, chunk):
        n = min(chunk, rows - at)
        r = np.arange(at, at + n)
        slots = table[r // page] * page + r % page
        assert len(set(slots.tolist())) == n                  # no two of a chunk's rows in one slot
        holds[slots] = r
        seen = np.flatnonzero(P.sees(n, at, rows, block, window, sinks).any(0))
        assert (holds[table[seen // page] * page + seen % page] == seen).all()
