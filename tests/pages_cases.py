"""Random page-pool states shared by the page operations' tests."""
import numpy as np


def state(rows, lens, num_pages, words, seed, width=None):
    """kv, table, lens, counts of requests with private pages in random places;
    every word of the pool is distinct enough to notice a wrong copy."""
    rng = np.random.default_rng(seed)
    need = [-(-n // 64) for n in lens]
    width = width or max(1, max(need, default=1))
    kv = rng.integers(-2**31, 2**31, (num_pages, 64, words), dtype=np.int64).astype(np.int32)
    table = np.full((rows, width), -1, np.int32)
    counts = np.zeros(num_pages, np.int32)
    perm = rng.permutation(num_pages)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        counts[perm[at:at + k]] = 1
        at += k
    assert at <= num_pages
    full = np.zeros(rows, np.int32)
    full[:len(lens)] = lens
    return kv, table, full, counts


def check_books(table, counts):
    """Every count is the number of table entries that name the page."""
    named = np.bincount(table[table >= 0], minlength=counts.size)
    np.testing.assert_array_equal(named, counts)
