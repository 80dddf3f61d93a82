"""The pair kernel (blocks of 128 rows) captured into graphs, on streams other
than the current one, from two threads at once, and with bad inputs; the same
for the kernel of 64-row blocks beside it."""
import threading

import pytest
import torch

import mla_paged_decode_gb300 as mla
from view_cases import SCALE, buffers, causal_seen, check, make, run_shared, run_window, window_seen

pytestmark = pytest.mark.gpu
WIDE = 2200     # block-table columns that send 128 rows and more to the pair kernel


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# heads: 64 leaves the requests' own pages to the other kernel, 128 takes them along
@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [64, 128])
def test_shared_replays_from_a_graph(kv_dtype, heads):
    lens = [700, 640, 900, 65, 0, 200]
    c = make(lens, heads, 1, kv_dtype, causal_seen(1), seed=100, shared=([0, 3, 6], [10, 1]), width=WIDE)
    out, lse = buffers(c)
    starts, pages = ints([0, 3, 6]), ints([10, 1])
    ws = mla.make_shared_workspace(c.q, c.kv, c.table, 2, c.kv_scale)
    run_shared(c, [0, 3, 6], [10, 1], ws=ws)        # kernels are loaded, limits raised
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.decode_shared(c.q, c.kv, c.table, c.lens, starts, pages, SCALE, 0, out, lse, kv_scale=c.kv_scale,
                          workspace=ws)
    g.replay()
    check(c, out, lse, what="replay")
    for new in ([701, 0, 641, 64, 1, 130], [0, 0, 0, 65, 0, 0], [640, 655, 900, 65, 66, 200]):
        # (no longer than the rows that were written)
        new = [min(a, b) for a, b in zip(new, lens)]
        c.lens.copy_(ints(new))
        c.seen = [[torch.arange(n)] for n in new]
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        g.replay()
        check(c, out, lse, what=f"replay {new}")
    assert mla.check_workspace(ws) == 0


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_window_replays_from_a_graph(kv_dtype):
    lens = [1000, 300, 64, 1] * 16
    c = make(lens, 128, 1, kv_dtype, window_seen(250, 70, 1), seed=101)
    c.kv = torch.where(torch.isnan(c.kv), 0, c.kv) if kv_dtype == "bf16" else torch.where(c.kv == 0x7F, 0, c.kv)
    for b, n in enumerate(lens):                    # every page of every request is there
        missing = (c.table[b] < 0).nonzero()[:, 0]
        c.table[b, missing[missing < -(-n // 64)]] = 0
    out, lse = buffers(c)
    ws = mla.make_workspace(c.q, c.kv, c.table, c.kv_scale)
    run_window(c, 250, 70, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.decode_window(c.q, c.kv, c.table, c.lens, 250, 70, SCALE, 0, out, lse, kv_scale=c.kv_scale, workspace=ws)
    g.replay()
    check(c, out, lse, what="replay")
    new = [999, 1, 0, 1] * 16
    c.lens.copy_(ints(new))
    seen = window_seen(250, 70, 1)
    c.seen = [[seen(n, 0)] for n in new]
    g.replay()
    check(c, out, lse, what="replay, shorter")
    assert mla.check_workspace(ws) == 0


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_on_another_stream(kv_dtype):
    s = torch.cuda.Stream()
    c = make([700, 640, 900], 128, 1, kv_dtype, causal_seen(1), seed=102, shared=([0, 3], [10]), width=WIDE)
    w = make([1000, 300, 64, 0] * 16, 128, 1, kv_dtype, window_seen(250, 3, 1), seed=103)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, wgot = run_shared(c, [0, 3], [10]), run_window(w, 250, 3)
    given = run_shared(c, [0, 3], [10], stream=s), run_window(w, 250, 3, stream=s)
    s.synchronize()
    check(c, *got)
    check(w, *wgot)
    for a, b in ((got, given[0]), (wgot, given[1])):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_from_two_threads(kv_dtype):
    """Each thread with its stream, buffers and workspaces: the same bits as alone."""
    cases = [make([700 + 64 * k, 640, 900], 128, 1, kv_dtype, causal_seen(1), seed=104 + k, shared=([0, 3], [10]),
                  width=WIDE) for k in range(2)]
    wcases = [make([1000 + k, 300, 64, 0] * 16, 128, 1, kv_dtype, window_seen(250, 3, 1), seed=106 + k)
              for k in range(2)]
    alone = [run_shared(c, [0, 3], [10]) for c in cases], [run_window(c, 250, 3) for c in wcases]
    got, errors = [None, None], []
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def work(k):
        try:
            with torch.cuda.stream(streams[k]):
                start.wait()
                for _ in range(20):
                    got[k] = run_shared(cases[k], [0, 3], [10]), run_window(wcases[k], 250, 3)
                streams[k].synchronize()
        except Exception as e:      # noqa: BLE001  (reported below, in the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for k in range(2):
        for a, b in zip((alone[0][k], alone[1][k]), got[k]):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# 16 heads: blocks of 64 rows; 64 at WIDE: shared pages on pairs, own pages in the
# other kernel; 128 at WIDE: both on pairs
@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,width", [(16, 0), (64, WIDE), (128, WIDE)])
@pytest.mark.parametrize("what", ["shared entry", "own entry", "negative entry", "length", "negative length", "starts",
                                  "pages", "negative pages"])
def test_bad_inputs_of_shared_are_reported(kv_dtype, heads, width, what):
    c = make([300, 200, 64], heads, 1, kv_dtype, causal_seen(1), seed=110, shared=([0, 3], [1]), width=width)
    starts, pages = [0, 3], [1]
    if what == "shared entry":
        c.table[:, 0] = c.kv.shape[0]
    if what == "own entry":
        c.table[1, 2] = c.kv.shape[0]
    if what == "negative entry":
        c.table[0, 3] = -7
    if what == "length":
        c.lens[2] = 64 * c.table.shape[1] + 1
    if what == "negative length":
        c.lens[2] = -1
    if what == "starts":
        starts = [0, 2]                       # the last request is in no group
    if what == "pages":
        pages = [c.table.shape[1] + 1]
    if what == "negative pages":
        pages = [-1]
    out, lse = buffers(c)
    ws = mla.make_shared_workspace(c.q, c.kv, c.table, 1, c.kv_scale)
    args = (c.q, c.kv, c.table, c.lens, ints(starts), ints(pages), SCALE, 0, out, lse)
    mla.decode_shared(*args, kv_scale=c.kv_scale, workspace=ws)
    assert mla.check_workspace(ws) == -9
    good = make([300, 200, 64], heads, 1, kv_dtype, causal_seen(1), seed=110, shared=([0, 3], [1]), width=width)
    check(good, *run_shared(good, [0, 3], [1], ws=ws), what="the same workspace afterwards")


@pytest.mark.parametrize("kv_dtype,copies", [("bf16", 1), ("bf16", 60), ("e4m3", 1)])
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("what", ["entry", "sink entry", "negative entry", "length", "negative length"])
def test_bad_inputs_of_window_are_reported(kv_dtype, copies, heads, what):
    lens = [300, 2000, 64] * copies
    c = make(lens, heads, 1, kv_dtype, window_seen(250, 70, 1), seed=111)
    if what == "entry":
        c.table[1, 30] = c.kv.shape[0]
    if what == "sink entry":
        c.table[1, 1] = 2**30
    if what == "negative entry":
        c.table[0, 3] = -7
    if what == "length":
        c.lens[2] = 64 * c.table.shape[1] + 1
    if what == "negative length":
        c.lens[2] = -5
    out, lse = buffers(c)
    ws = mla.make_workspace(c.q, c.kv, c.table, c.kv_scale)
    mla.decode_window(c.q, c.kv, c.table, c.lens, 250, 70, SCALE, 0, out, lse, kv_scale=c.kv_scale, workspace=ws)
    assert mla.check_workspace(ws) == -9
    good = make(lens, heads, 1, kv_dtype, window_seen(250, 70, 1), seed=111)
    check(good, *run_window(good, 250, 70, ws=ws), what="the same workspace afterwards")
