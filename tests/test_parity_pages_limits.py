"""Page operations at the ends of their ranges: sinks, windows and lengths up to
2^31 - 1."""
import numpy as np
import pytest
import torch

import mla_paged_decode_gb300 as mla
from oracle import pages_oracle as po
from pages_cases import state

pytestmark = pytest.mark.gpu
TOP = 2**31 - 1


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("window,sinks", [(100, TOP), (100, TOP - 63), (100, TOP - 62), (TOP, 0), (TOP, TOP), (1, TOP - 1)])
def test_free_keeps_what_the_largest_views_see(window, sinks):
    host = list(state(4, [640, 65, 1, 500], 40, 3, seed=70))
    _, table, lens, counts = (torch.from_numpy(x.copy()).cuda() for x in host)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = np.array([640, 65, 1, 200])
    mla.pages_free(table, lens, counts, ints(new), window=window, sinks=sinks, error_word=err)
    assert po.free(*host[1:], new, window, sinks) == 0 == int(err.item())
    for got, want in zip((table, lens, counts), host[1:]):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_free_and_alloc_of_the_longest_request():
    """A table of 2^25 pages holds every length below 2^31."""
    width = 2**25
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, width - 2] = 2, 0
    counts = ints([1, 0, 1, 0])
    lens = ints([TOP - 64])                 # 2^25 - 1 pages
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.pages_alloc(table, lens, counts, ints([TOP]), error_word=err)
    assert table[0, width - 1].item() == 1 and counts.tolist() == [1, 1, 1, 0]
    lens.fill_(TOP)
    mla.pages_free(table, lens, counts, ints([TOP]), error_word=err)
    assert table[0, [0, width - 2, width - 1]].tolist() == [2, 0, 1] and counts.tolist() == [1, 1, 1, 0]
    mla.pages_free(table, lens, counts, ints([TOP]), window=1, sinks=1, error_word=err)
    assert table[0, [0, width - 2, width - 1]].tolist() == [2, -1, 1] and counts.tolist() == [0, 1, 1, 0]
    mla.pages_free(table, lens, counts, ints([TOP - 64]), error_word=err)
    assert table[0, [0, width - 2, width - 1]].tolist() == [2, -1, -1] and counts.tolist() == [0, 0, 1, 0]
    assert lens.item() == TOP - 64 and err.item() == 0


def test_alloc_of_more_pages_than_32_bits_count():
    """64 requests ask for 2^25 pages each: the ranks of those behind them pass
    2^31.  Only the first one, which asks for two, fits."""
    rows, width = 67, 2**25                 # a table of 9 GB
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    counts = torch.zeros(3000, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.pages_alloc(table, lens, counts, ints([65] + [TOP] * 64 + [1, TOP]), error_word=err)
    assert err.item() == mla.PAGES_FULL
    assert table[0, :3].tolist() == [0, 1, -1] and int(counts.sum()) == 2
    assert (table[0, 2:] == -1).all() and (table[1:] == -1).all()


@pytest.mark.parametrize("pages", [30, 5000])
def test_compact_reports_entries_of_free_pages_below_the_live_ones(pages):
    """The page is free, something moves into it, and the entry stays as it is."""
    host = list(state(4, [640, 640, 64], pages, 144, seed=71))
    po.free(*host[1:], np.array([640, 0, 64, 0]))
    n = int((host[3] > 0).sum())
    hole = 0 if host[3][0] == 0 else int(np.flatnonzero(host[3] == 0)[0])
    assert hole < n
    host[1][3, :2] = [hole, -1]
    kv, table, counts = (torch.from_numpy(host[i].copy()).cuda() for i in (0, 1, 3))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.pages_compact(kv.view(torch.uint8).view(pages, 64, 576), table, counts, error_word=err)
    assert po.compact(host[0], host[1], host[3])[0] == po.BAD and host[1][3, 0] == hole
    assert err.item() == mla.PAGES_BAD_ENTRY
    for got, want in zip((kv, table, counts), (host[0], host[1], host[3])):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("entry", [-2, -2**31, 40, TOP])
def test_fork_reports_any_entry_that_is_no_page(entry):
    host = list(state(4, [300, 64], 40, 288, seed=72))
    host[1][0, 1] = entry
    kv, table, lens, counts = (torch.from_numpy(x.copy()).cuda() for x in host)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    parents, children = np.array([0, 1]), np.array([2, 3])
    mla.pages_fork(kv.view(torch.bfloat16), table, lens, counts, ints(parents), ints(children), error_word=err)
    assert po.fork(*host, parents, children) == po.BAD == err.item()
    assert host[1][2, 1] == -1
    for got, want in zip((kv, table, lens, counts), host):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
