"""What the page operations' oracle says about table entries that name no live page."""
import numpy as np

from oracle import pages_oracle as po
from pages_cases import state


def test_compact_reports_an_entry_of_a_free_page_wherever_it_lies():
    for at in ("below", "past"):
        kv, table, lens, counts = state(4, [640, 640, 64], 30, 3, seed=5)
        po.free(table, lens, counts, np.array([640, 0, 64, 0]))
        n = int((counts > 0).sum())
        free = np.flatnonzero(counts == 0)
        stray = int(free[free < n][0] if at == "below" else free[free >= n][0])
        table[3, 0] = stray
        others = table[:3].copy()
        pages = {int(p): kv[p].copy() for p in others[others >= 0]}
        err, remap, *_ = po.compact(kv, table, counts)
        assert err == po.BAD and table[3, 0] == stray
        for before, after in zip(others[others >= 0], table[:3][others >= 0]):
            assert remap[before] == after
            np.testing.assert_array_equal(kv[after], pages[int(before)])


def test_fork_reports_any_entry_that_is_no_page():
    for entry in (-2, -2**31, 40, 2**31 - 1):
        kv, table, lens, counts = state(4, [300, 64], 40, 3, seed=6)
        table[0, 1] = entry
        assert po.fork(kv, table, lens, counts, np.array([0, 1]), np.array([2, 3])) == po.BAD
        assert table[2, 1] == -1 and lens[2] == 300 and table[3, 0] == table[1, 0]
