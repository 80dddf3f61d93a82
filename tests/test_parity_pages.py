"""GPU parity of the page operations with their oracle: pools, tables,
lengths, counts and remaps equal word for word, bad entries skipped and
reported, a full pool reported, and graph replay."""
import numpy as np
import pytest
import torch

import mla_paged_decode_gb300 as mla
from oracle import pages_oracle as po
from pages_cases import check_books, state

pytestmark = pytest.mark.gpu
WORDS = {"bf16": 288, "e4m3": 144}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


class Pool:
    """The same state on the host (oracle) and on the device."""

    def __init__(self, rows, lens, num_pages, kv_dtype, seed, width=None):
        self.host = list(state(rows, lens, num_pages, WORDS[kv_dtype], seed, width))
        self.dtype = torch.bfloat16 if kv_dtype == "bf16" else torch.uint8
        self.up()

    def up(self):
        kv, table, lens, counts = (torch.from_numpy(x.copy()).cuda() for x in self.host)
        self.kv, self.table, self.lens, self.counts = kv.view(self.dtype), table, lens, counts
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def check(self, err, books=True):
        torch.cuda.synchronize()
        for got, want, name in zip((self.kv.view(torch.int32), self.table, self.lens, self.counts),
                                   self.host, ("kv", "table", "lens", "counts")):
            np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)
        assert int(self.err.item()) == err
        if books:
            check_books(self.host[1], self.host[3])


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,pages", [([1], 5), ([64], 5), ([63, 64, 65, 0, 200, 129], 40),
                                        (list(range(1, 400, 7)), 2500)])
def test_fork(kv_dtype, lens, pages):
    n = len(lens)
    p = Pool(4 * n + 3, lens, pages, kv_dtype, seed=n)
    rng = np.random.default_rng(n)
    parents = rng.integers(0, n, 3 * n)
    children = n + rng.permutation(3 * n + 3)[:3 * n]
    mla.pages_fork(p.kv, p.table, p.lens, p.counts, ints(parents), ints(children), error_word=p.err)
    p.check(po.fork(*p.host, parents, children))


def test_fork_reports_bad_entries_and_a_full_pool():
    p = Pool(12, [100, 30, 65, 128], 9, "bf16", seed=3)
    p.host[1][1, 0] = 77                    # the partial page of request 1
    p.host[2][3] = 64 * p.host[1].shape[1] + 1  # a length past the table
    p.up()
    parents, children = np.array([0, 1, -1, 3, 0, 2, 0]), np.array([5, 6, 7, 8, 12, 9, 10])
    mla.pages_fork(p.kv, p.table, p.lens, p.counts, ints(parents), ints(children), error_word=p.err)
    p.check(po.fork(*p.host, parents, children), books=False)
    # three pages are free: the fourth fork of a partial page finds none
    p = Pool(12, [100], 5, "e4m3", seed=4)
    parents, children = np.zeros(5, int), np.arange(3, 8)
    mla.pages_fork(p.kv, p.table, p.lens, p.counts, ints(parents), ints(children), error_word=p.err)
    assert po.fork(*p.host, parents, children) == po.FULL
    p.check(po.FULL)


@pytest.mark.parametrize("rows,pages", [(1, 3), (5, 64), (300, 6000)])
def test_alloc(rows, pages):
    rng = np.random.default_rng(rows)
    lens = rng.integers(0, min(600, 32 * pages // rows), rows).tolist()
    p = Pool(rows, lens, pages, "e4m3", seed=rows, width=40)
    new = np.minimum(np.array(lens) + rng.integers(-20, 900, rows).clip(0), 2560)
    mla.pages_alloc(p.table, p.lens, p.counts, ints(new), error_word=p.err)
    p.check(po.alloc(*p.host[1:], new))


def test_alloc_reports_what_does_not_fit():
    p = Pool(4, [64, 64, 64, 64], 8, "e4m3", seed=1, width=4)
    new = np.array([128, 257, 192, 256])    # past the table; fits; does not fit
    mla.pages_alloc(p.table, p.lens, p.counts, ints(new), error_word=p.err)
    want = po.alloc(*p.host[1:], new)
    assert want == po.BAD | po.FULL
    p.check(want)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 5), (128, 64), (64, 65), (10000, 0)])
def test_free(window, sinks):
    lens = [0, 1, 63, 64, 65, 500, 640, 129, 1000]
    p = Pool(11, lens, 80, "e4m3", seed=window + sinks)
    po.fork(*p.host, np.array([6]), np.array([10]))   # shared pages among them
    p.up()
    new = np.array([0, 0, 63, 1, 65, 200, 640, 128, 1000, 0, 0])
    mla.pages_free(p.table, p.lens, p.counts, ints(new), window=window, sinks=sinks, error_word=p.err)
    p.check(po.free(*p.host[1:], new, window, sinks))


def test_free_reports_growth_and_double_frees():
    p = Pool(3, [100, 100, 64], 9, "e4m3", seed=2)
    p.host[3][p.host[1][1, 0]] = 0          # already free
    p.host[1][2, 0] = 50                    # no such page
    p.up()
    new = np.array([101, 0, 0])
    mla.pages_free(p.table, p.lens, p.counts, ints(new), error_word=p.err)
    assert po.free(*p.host[1:], new) == po.BAD
    p.check(po.BAD, books=False)


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,pages", [(1, 1), (3, 7), (40, 1024), (40, 1025), (150, 3001)])
def test_compact(kv_dtype, rows, pages):
    rng = np.random.default_rng(pages)
    lens = rng.integers(1, max(2, 48 * pages // rows), rows).tolist()
    p = Pool(rows, lens, pages, kv_dtype, seed=pages)
    po.free(*p.host[1:], np.where(rng.random(rows) < 0.5, 0, p.host[2]))
    p.up()
    remap = torch.full((pages,), 99, dtype=torch.int32, device="cuda")
    totals = mla.pages_compact(p.kv, p.table, p.counts, remap=remap, error_word=p.err)
    err, want, n, m = po.compact(p.host[0], p.host[1], p.host[3])
    p.check(err)
    np.testing.assert_array_equal(remap.cpu().numpy(), want)
    assert totals[:8].view(torch.int32).tolist() == [n, m]


@pytest.mark.parametrize("live", ["none", "all"])
def test_compact_of_an_empty_and_of_a_full_pool(live):
    p = Pool(2, [] if live == "none" else [64 * 9, 64 * 7 - 3], 16, "e4m3", seed=5, width=9)
    mla.pages_compact(p.kv, p.table, p.counts, error_word=p.err)
    po.compact(p.host[0], p.host[1], p.host[3])
    p.check(0)


def test_compact_skips_entries_of_no_live_page():
    p = Pool(3, [640, 64], 30, "e4m3", seed=6)
    n = int((p.host[3] > 0).sum())
    stray = [q for q in range(n, 30) if p.host[3][q] == 0][0]
    p.host[1][2, :3] = [stray, 30, -5]
    p.up()
    mla.pages_compact(p.kv, p.table, p.counts, error_word=p.err)
    assert po.compact(p.host[0], p.host[1], p.host[3])[0] == po.BAD
    p.check(po.BAD, books=False)


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 200])
def test_copy_between_and_within_pools(kv_dtype, n):
    a, b = Pool(1, [], 500, kv_dtype, seed=n), Pool(1, [], 300, kv_dtype, seed=n + 1)
    rng = np.random.default_rng(n)
    src, dst = rng.permutation(500)[:n], rng.permutation(300)[:n]
    src[0] = 500 if n > 1 else src[0]       # one bad entry
    mla.pages_copy(a.kv, b.kv, ints(src), ints(dst), error_word=b.err)
    b.check(po.copy(a.host[0], b.host[0], src, dst))
    src = rng.permutation(500)
    src, dst = src[:n], src[n:2 * n]        # disjoint
    mla.pages_copy(a.kv, a.kv, ints(src), ints(dst), error_word=a.err)
    a.check(po.copy(a.host[0], a.host[0], src, dst))


def test_empty_calls_do_nothing():
    p = Pool(3, [100], 9, "bf16", seed=8)
    none = ints(np.zeros(0, int))
    mla.pages_fork(p.kv, p.table, p.lens, p.counts, none, none, error_word=p.err)
    mla.pages_copy(p.kv, p.kv, none, none, error_word=p.err)
    mla.pages_free(p.table, p.lens, p.counts, p.lens.clone(), error_word=p.err)
    mla.pages_alloc(p.table, p.lens, p.counts, p.lens.clone(), error_word=p.err)
    p.check(0)


def test_a_captured_step_replays():
    """fork, free and compact captured on one stream; each replay works on
    what the buffers then hold."""
    p = Pool(9, [100, 300, 64], 40, "bf16", seed=11)
    start = [x.copy() for x in p.host]
    parents, children = np.array([0, 1, 1]), np.array([4, 5, 7])
    keep = np.array([100, 0, 64, 0, 90, 300, 0, 300, 0])
    dp, dc, dk = ints(parents), ints(children), ints(keep)
    ws = mla.make_pages_workspace(p.counts)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.pages_fork(p.kv, p.table, p.lens, p.counts, dp, dc, workspace=ws, error_word=p.err)
        mla.pages_free(p.table, p.lens, p.counts, dk, error_word=p.err)
        mla.pages_compact(p.kv, p.table, p.counts, workspace=ws, error_word=p.err)
    for seed in (0, 1):
        for t, x in zip((p.kv.view(torch.int32), p.table, p.lens, p.counts), start):
            t.copy_(torch.from_numpy(x))
        if seed:
            dp.copy_(torch.tensor([2, 0, 1]))
            parents = np.array([2, 0, 1])
            dk.copy_(ints([10, 0, 64, 0, 64, 100, 0, 1, 0]))
            keep = np.array([10, 0, 64, 0, 64, 100, 0, 1, 0])
        p.host = [x.copy() for x in start]
        g.replay()
        po.fork(*p.host, parents, children)
        po.free(*p.host[1:], keep)
        po.compact(p.host[0], p.host[1], p.host[3])
        p.check(0)


def test_calls_run_on_the_given_stream():
    p = Pool(6, [300, 100], 40, "bf16", seed=12)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    parents, children = np.array([0, 1]), np.array([3, 4])
    mla.pages_fork(p.kv, p.table, p.lens, p.counts, ints(parents), ints(children), error_word=p.err, stream=s)
    s.synchronize()
    p.check(po.fork(*p.host, parents, children))
