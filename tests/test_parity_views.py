"""GPU parity of decode_window and decode_shared with their definition in 64
bits: windows and sinks from one token to longer than the request, groups of
every size, head counts that leave blocks part full, several query tokens,
empty requests, both cache types, NaN in every row out of view."""
import math

import pytest
import torch

import mla_paged_decode_gb300 as mla
from view_cases import (buffers, causal_seen, check, make, run_shared, run_window, window_seen)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


LENS = [1, 2, 63, 64, 65, 128, 300, 0, 777]


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,q_len", [(16, 1), (64, 1), (1, 1), (20, 3), (128, 2), (7, 16), (65, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 4), (64, 0), (65, 64), (130, 70), (10**9, 3), (100, 2**31 - 1)])
def test_window(kv_dtype, heads, q_len, window, sinks):
    c = make(LENS, heads, q_len, kv_dtype, window_seen(window, sinks, q_len), seed=heads + window % 1000)
    base = heads % 2
    out, lse = run_window(c, window, sinks, base)
    check(c, out, lse, base, f"window {window} sinks {sinks}")


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,q_len", [(128, 1), (65, 2), (100, 2), (16, 16), (80, 5), (96, 3)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 4), (70, 0), (64, 64), (130, 70), (300, 200), (10**9, 3), (100, 2**31 - 1)])
def test_window_of_many_rows(kv_dtype, heads, q_len, window, sinks):
    """Blocks of 128 rows, whole and part full; windows that start and end in
    every part of a page and of a tile of four (a bf16 cache takes them when
    there are enough rows)."""
    lens = (LENS + [256, 257, 321, 1000, 1003, 1041]) * (4 if kv_dtype == "bf16" else 1)
    c = make(lens, heads, q_len, kv_dtype, window_seen(window, sinks, q_len), seed=heads + window % 1000)
    base = heads % 2
    out, lse = run_window(c, window, sinks, base)
    check(c, out, lse, base, f"window {window} sinks {sinks}")


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_window_of_many_rows_over_many_and_long_requests(kv_dtype):
    lens = [9000, 4096, 12001, 8191]
    c = make(lens, 128, 2, kv_dtype, window_seen(2500, 40, 2), seed=6)
    check(c, *run_window(c, 2500, 40), what="long")
    c = make([20000], 128, 1, kv_dtype, window_seen(16000, 0, 1), seed=7)
    check(c, *run_window(c, 16000, 0), what="one")
    c = make([(37 * b) % 300 for b in range(410)], 65, 2, kv_dtype, window_seen(90, 5, 2), seed=8)
    check(c, *run_window(c, 90, 5), what="many")


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_window_over_long_requests(kv_dtype):
    lens = [9000, 4096, 12001, 8191]
    c = make(lens, 64, 1, kv_dtype, window_seen(2500, 40, 1), seed=3)
    check(c, *run_window(c, 2500, 40), what="long")


def test_window_of_the_whole_request_is_the_plain_decode():
    """Both meet the definition; a request of one tile, which no split and no
    merge weight touches, has the same bits."""
    c = make(LENS, 64, 1, "bf16", causal_seen(1), seed=5)
    out, lse = run_window(c, 4096, 0)
    o2, l2 = buffers(c)
    mla.decode_partial(c.q, c.kv, c.table, c.lens, 0, 1, 1 / math.sqrt(192.0), 0, o2, l2)
    check(c, out, lse, what="window")
    one_tile = c.lens <= 64
    assert int(one_tile.sum()) >= 4 and torch.equal(out[one_tile], o2[one_tile])


GROUPS = [
    # lens, group_starts, shared_pages
    ([300], [0, 1], [4]),
    ([65, 70, 64, 129], [0, 4], [1]),
    ([200, 130, 131, 500, 64, 64, 1, 0], [0, 3, 3, 5, 8], [2, 7, 1, 0]),
    ([640 + k for k in range(1, 22)], [0, 1, 21], [10, 9]),
    ([10, 400, 100, 0], [0, 4], [3]),          # shorter than the shared pages
    ([512] * 3, [0, 3], [8]),                  # no tail
]


# A wide block table, whose rows x tokens bound the work, takes a bf16 cache's
# groups of 128 rows and more to the pair kernel.
WIDE = 2200


@pytest.mark.parametrize("kv_dtype,width", [("bf16", 0), ("bf16", WIDE), ("e4m3", 0), ("e4m3", WIDE)])
@pytest.mark.parametrize("heads,q_len", [(16, 1), (64, 1), (1, 1), (20, 3), (128, 2), (7, 16), (65, 1)])
@pytest.mark.parametrize("group", range(len(GROUPS)))
def test_shared(kv_dtype, width, heads, q_len, group):
    lens, starts, pages = GROUPS[group]
    c = make(lens, heads, q_len, kv_dtype, causal_seen(q_len), seed=heads + group, shared=(starts, pages),
             width=width)
    base = group % 2
    out, lse = run_shared(c, starts, pages, base)
    check(c, out, lse, base, f"group {group}")


@pytest.mark.parametrize("kv_dtype,width", [("bf16", 0), ("bf16", WIDE), ("e4m3", 0), ("e4m3", WIDE)])
@pytest.mark.parametrize("n,heads,pages,q_len", [(40, 16, 70, 1), (9, 128, 200, 1), (3, 64, 301, 2), (33, 40, 50, 1)])
def test_shared_long_prefix(kv_dtype, width, n, heads, pages, q_len):
    lens = [64 * pages + (37 * b) % 300 for b in range(n)]
    c = make(lens, heads, q_len, kv_dtype, causal_seen(q_len), seed=n, shared=([0, n], [pages]), width=width)
    check(c, *run_shared(c, [0, n], [pages]), what="long prefix")


@pytest.mark.parametrize("kv_dtype,width", [("bf16", 0), ("bf16", WIDE), ("e4m3", 0), ("e4m3", WIDE)])
def test_shared_with_more_requests_than_threads(kv_dtype, width):
    """Hundreds of requests and groups, empty groups among them: the schedule
    walks them in chunks; the last group is large."""
    starts, pages = [0], []
    for k in range(90):
        starts.append(starts[-1] + k % 4)
        pages.append(k % 3)
    starts.append(starts[-1] + 330)
    pages.append(5)
    lens = [64 * pages[k] + (13 * b) % 150 for k in range(len(pages)) for b in range(starts[k], starts[k + 1])]
    c = make(lens, 40, 1, kv_dtype, causal_seen(1), seed=21, shared=(starts, pages), width=width)
    check(c, *run_shared(c, starts, pages), what="many requests")


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_window_with_more_requests_than_threads(kv_dtype):
    lens = [(37 * b) % 300 for b in range(410)]
    c = make(lens, 20, 1, kv_dtype, window_seen(90, 5, 1), seed=22)
    check(c, *run_window(c, 90, 5), what="many requests")


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("gain", [0.0, 40.0])
def test_flat_and_steep_scores(kv_dtype, gain):
    """All scores zero; one token taking nearly all the weight."""
    c = make([1000, 65, 300], 16, 1, kv_dtype, window_seen(500, 3, 1), seed=23, q_gain=gain)
    check(c, *run_window(c, 500, 3), what="window")
    c = make([1000, 1001, 1090], 64, 1, kv_dtype, causal_seen(1), seed=24, shared=([0, 3], [15]), q_gain=gain,
             width=WIDE)
    check(c, *run_shared(c, [0, 3], [15]), what="shared")


@pytest.mark.parametrize("width", [0, WIDE])
def test_a_query_that_is_not_finite_stays_in_its_row(width):
    c = make([700, 640, 655], 64, 1, "bf16", causal_seen(1), seed=25, shared=([0, 3], [9]), width=width)
    good, glse = run_shared(c, [0, 3], [9])
    c.q[1, 0, 7, 3] = math.nan
    c.q[2, 0, 60, 570] = math.inf
    out, lse = run_shared(c, [0, 3], [9])
    rest = torch.ones(3, 1, 64, dtype=torch.bool)
    rest[1, 0, 7] = rest[2, 0, 60] = False
    assert torch.isfinite(out[rest]).all()
    assert (out[rest].float() - good[rest].float()).abs().max() <= 2.0**-7 * good.float().abs().max()
    assert not torch.isfinite(out[1, 0, 7].float()).all()


@pytest.mark.parametrize("kv_dtype,width", [("bf16", 0), ("bf16", WIDE), ("e4m3", 0), ("e4m3", WIDE)])
def test_shared_scores_of_a_wide_range(kv_dtype, width):
    """Running maxima that grow across tiles and rows whose weights sit on few tokens."""
    lens = [64 * 30 + 17] * 6
    c = make(lens, 64, 1, kv_dtype, causal_seen(1), seed=8, shared=([0, 6], [30]), q_gain=6.0, width=width)
    check(c, *run_shared(c, [0, 6], [30]), what="wide scores")


@pytest.mark.parametrize("kv_dtype,width", [("bf16", 0), ("bf16", WIDE), ("e4m3", 0), ("e4m3", WIDE)])
def test_results_repeat_bit_for_bit_and_workspaces_are_reusable(kv_dtype, width):
    lens = [64 * 40 + 100 * b for b in range(9)]
    c = make(lens, 64, 1, kv_dtype, causal_seen(1), seed=4, shared=([0, 4, 9], [40, 40]), width=width)
    ws = mla.make_shared_workspace(c.q, c.kv, c.table, 2, c.kv_scale)
    first = run_shared(c, [0, 4, 9], [40, 40], ws=ws)
    for _ in range(3):
        again = run_shared(c, [0, 4, 9], [40, 40], ws=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_views_replay_from_a_graph_with_new_lengths():
    c = make([500, 300], 16, 1, "bf16", window_seen(100, 4, 1), seed=6)
    full = make([500, 300], 16, 1, "bf16", causal_seen(1), seed=6, shared=([0, 2], [2]))
    out, lse = buffers(c)
    so, sl = buffers(full)
    ws = mla.make_workspace(c.q, c.kv, c.table)
    sws = mla.make_shared_workspace(full.q, full.kv, full.table, 1)
    starts = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    pages = torch.tensor([2], dtype=torch.int32, device="cuda")
    run_window(c, 100, 4, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.decode_window(c.q, c.kv, c.table, c.lens, 100, 4, 1 / math.sqrt(192.0), 0, out, lse, workspace=ws)
        mla.decode_shared(full.q, full.kv, full.table, full.lens, starts, pages, 1 / math.sqrt(192.0), 0, so, sl,
                          workspace=sws)
    g.replay()
    check(c, out, lse, what="replay")
    check(full, so, sl, what="replay")
    full.lens.copy_(torch.tensor([400, 129], dtype=torch.int32))
    full.seen = [[torch.arange(400)], [torch.arange(129)]]
    g.replay()
    check(full, so, sl, what="replay, shorter")


def test_views_on_another_stream():
    s = torch.cuda.Stream()
    c = make(LENS, 16, 1, "bf16", window_seen(70, 3, 1), seed=7)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = run_window(c, 70, 3)
    s.synchronize()
    check(c, out, lse)


@pytest.mark.parametrize("what", ["entry", "length", "starts", "pages"])
def test_bad_inputs_are_reported(what):
    lens = [300, 200, 64]
    c = make(lens, 16, 1, "bf16", causal_seen(1), seed=9, shared=([0, 3], [1]))
    starts, pages = [0, 3], [1]
    if what == "entry":
        c.table[1, 2] = c.kv.shape[0]
    if what == "length":
        c.lens[2] = 64 * c.table.shape[1] + 1
    if what == "starts":
        starts = [0, 2]                       # the last request is in no group
    if what == "pages":
        pages = [c.table.shape[1] + 1]
    out, lse = buffers(c)
    ws = mla.make_shared_workspace(c.q, c.kv, c.table, 1)
    mla.decode_shared(c.q, c.kv, c.table, c.lens, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                      torch.tensor(pages, dtype=torch.int32, device="cuda"), 0.1, 0, out, lse, workspace=ws)
    assert mla.check_workspace(ws) == -9
    if what in ("entry", "length"):
        ws = mla.make_workspace(c.q, c.kv, c.table)
        mla.decode_window(c.q, c.kv, c.table, c.lens, 10**6, 0, 0.1, 0, out, lse, workspace=ws)
        assert mla.check_workspace(ws) == -9


def test_a_pool_past_4_gib():
    """Page numbers whose byte offsets pass 32 bits."""
    pages = 62000                                  # 4.6 GB of bf16 rows
    small = make([500, 640], 64, 1, "bf16", causal_seen(1), seed=31, shared=([0, 2], [7]))
    n = small.kv.shape[0]
    kv = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(n, dtype=torch.int32, device="cuda") + (pages - n)
    mla.pages_copy(small.kv, kv, torch.arange(n, dtype=torch.int32, device="cuda"), at)
    small.kv = kv
    small.table = torch.where(small.table >= 0, small.table + (pages - n), small.table)
    check(small, *run_shared(small, [0, 2], [7]), what="shared")
    full = small.seen
    check(small, *run_window(small, 10**6, 0), what="window")
    pad = torch.full((2, WIDE), -1, dtype=torch.int32, device="cuda")
    pad[:, :small.table.shape[1]] = small.table
    small.table = pad
    small.q = small.q.repeat(1, 2, 1, 1).contiguous()       # two query tokens: 128 rows a request
    small.seen = [[s[0][:-1], s[0]] for s in full]
    check(small, *run_shared(small, [0, 2], [7]), what="shared, pairs")
