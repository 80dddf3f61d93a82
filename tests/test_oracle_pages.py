"""The page operations' oracle on hand-worked states, and the books it keeps:
after any sequence of operations every reference count is the number of table
entries that name the page, and a request reads the rows it wrote."""
import numpy as np

from oracle import pages_oracle as po
from pages_cases import check_books, state


def test_fork_shares_full_pages_and_copies_the_partial_one():
    kv, table, lens, counts = state(4, [130], 6, 3, seed=0)
    row = table[0].copy()
    before = kv.copy()
    free = np.flatnonzero(counts == 0)
    assert po.fork(kv, table, lens, counts, np.array([0, 0]), np.array([2, 1])) == 0
    assert table[2].tolist() == [row[0], row[1], free[0]] and table[1].tolist() == [row[0], row[1], free[1]]
    assert lens.tolist() == [130, 130, 130, 0]
    assert counts[row[0]] == counts[row[1]] == 3 and counts[row[2]] == 1
    np.testing.assert_array_equal(kv[free[0], :2], before[row[2], :2])
    np.testing.assert_array_equal(kv[free[0], 2:], before[free[0], 2:])
    check_books(table, counts)


def test_fork_without_room_leaves_an_empty_child():
    kv, table, lens, counts = state(3, [65], 2, 3, seed=1)
    assert po.fork(kv, table, lens, counts, np.array([0]), np.array([1])) == po.FULL
    assert lens[1] == 0 and (table[1] == -1).all()
    check_books(table, counts)


def test_alloc_takes_the_lowest_pages_in_request_order():
    kv, table, lens, counts = state(3, [64, 1, 0], 8, 3, seed=2, width=3)
    free = np.flatnonzero(counts == 0)
    assert po.alloc(table, lens, counts, np.array([65, 64, 128])) == 0
    assert table[0, 1] == free[0] and table[2, :2].tolist() == free[1:3].tolist()
    assert table[1].tolist()[1:] == [-1, -1]
    check_books(table, counts)


def test_free_trims_to_the_window():
    kv, table, lens, counts = state(1, [640], 12, 3, seed=3)
    # the next query (position 640) sees t > 512 and t < 70: pages 0, 1 and 8, 9
    po.free(table, lens, counts, np.array([640]), window=128, sinks=70)
    assert [i for i in range(10) if table[0, i] >= 0] == [0, 1, 8, 9]
    check_books(table, counts)


def test_compact_moves_the_tail_into_the_holes():
    kv, table, lens, counts = state(5, [100, 64, 200, 10, 640], 40, 3, seed=4)
    before = [kv[table[b][table[b] >= 0]].copy() for b in range(5)]
    po.free(table, lens, counts, np.array([100, 0, 200, 0, 640]))
    err, remap, n, m = po.compact(kv, table, counts)
    assert err == 0 and (counts[:n] > 0).all() and (counts[n:] == 0).all()
    for b in (0, 2, 4):
        np.testing.assert_array_equal(kv[table[b][table[b] >= 0]], before[b])
    check_books(table, counts)


def test_books_hold_over_a_random_sequence():
    rng = np.random.default_rng(9)
    kv, table, lens, counts = state(12, [300, 77, 5], 200, 2, seed=9, width=8)
    for _ in range(60):
        live, dead = np.flatnonzero(lens > 0), np.flatnonzero(lens == 0)
        if live.size and dead.size and rng.random() < 0.5:
            po.fork(kv, table, lens, counts, rng.choice(live, 1), rng.choice(dead, 1))
        else:
            keep = np.where(rng.random(12) < 0.15, 0, lens)
            po.free(table, lens, counts, keep)
        new = np.where(lens > 0, np.minimum(lens + rng.integers(0, 90, 12), 512), 0)
        if po.alloc(table, lens, counts, new) == 0:
            lens[:] = new
        check_books(table, counts)
    po.compact(kv, table, counts)
    check_books(table, counts)
