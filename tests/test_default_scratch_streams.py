"""Calls on a stream that is behind, without a workspace or outputs of the
caller's: what the binding allocates stays theirs until that stream has run
them, whatever the current stream allocates and fills meanwhile."""

import numpy as np
import pytest
import torch

import mla_paged_decode_gb300 as mla
from oracle import pages_oracle as po
from pages_cases import check_books, state
from view_cases import SCALE, buffers, causal_seen, check, make, window_seen

pytestmark = pytest.mark.gpu
BEHIND = 1_000_000_000      # clocks: about half a second of waiting in front of the call


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


def behind(call, sizes, warm=None):
    """Runs call(stream) on a stream that is kept waiting, while the current
    stream allocates and fills blocks of the sizes that the call may have used.
    (The call, or one like it, has run before: loading kernels may wait.)"""
    (warm or call)(None)
    s = torch.cuda.Stream()
    for n in sizes:             # blocks of these sizes are in both streams' pools
        torch.empty(n, dtype=torch.uint8, device="cuda")
        with torch.cuda.stream(s):
            torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BEHIND)
    r = call(s)
    assert not s.query(), "the stream was not behind"
    junk = [torch.full((n,), 0x7B, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.current_stream().synchronize()
    s.synchronize()
    del junk
    return r


@pytest.mark.parametrize("heads", [16, 128])
def test_decode_window(heads):
    c = make([900, 64, 1, 0] * 8, heads, 1, "e4m3", window_seen(300, 70, 1), seed=50)
    out, lse = buffers(c)
    n = mla.workspace_size(c.q, c.kv, c.table, c.kv_scale)
    behind(lambda s: mla.decode_window(c.q, c.kv, c.table, c.lens, 300, 70, SCALE, 0, out, lse, kv_scale=c.kv_scale,
                                       stream=s), [n])
    check(c, out, lse)


@pytest.mark.parametrize("width", [0, 2200])
def test_decode_shared(width):
    c = make([700, 690, 801, 640], 64, 1, "bf16", causal_seen(1), seed=51, shared=([0, 4], [10]), width=width)
    out, lse = buffers(c)
    starts = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    pages = torch.tensor([10], dtype=torch.int32, device="cuda")
    n = mla.make_shared_workspace(c.q, c.kv, c.table, 1).numel()
    behind(lambda s: mla.decode_shared(c.q, c.kv, c.table, c.lens, starts, pages, SCALE, 0, out, lse, stream=s), [n])
    check(c, out, lse)


def test_decode_partial_and_dcp():
    c = make([5000, 64, 1, 0], 64, 1, "bf16", causal_seen(1), seed=52)
    want, want_lse = buffers(c)
    mla.decode_partial(c.q, c.kv, c.table, c.lens, 0, 1, SCALE, 0, want, want_lse)
    out, lse = buffers(c)
    n = mla.workspace_size(c.q, c.kv, c.table)
    behind(lambda s: mla.decode_partial(c.q, c.kv, c.table, c.lens, 0, 1, SCALE, 0, out, lse, stream=s), [n])
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    want, _, parts, plses = mla.decode_dcp(c.q, c.kv, c.table, c.lens, 4, SCALE, 0)
    n = mla.make_dcp_workspace(c.q, c.kv, c.table, 4).numel()
    sizes = [n, want.numel() * 2, parts.numel() * 2, plses.numel() * 4]
    got, _, gparts, glses = behind(lambda s: mla.decode_dcp(c.q, c.kv, c.table, c.lens, 4, SCALE, 0, stream=s), sizes)
    assert torch.equal(got, want) and torch.equal(gparts, parts) and torch.equal(glses, plses)


def test_dcp_local_metadata():
    lens = torch.tensor([1000, 3, 0], dtype=torch.int32, device="cuda")
    idx = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    slots = torch.arange(3 * 1024, dtype=torch.int32, device="cuda").view(3, 1024)
    want = mla.dcp_local_metadata(lens, idx, slots, 1, 2, max_pages=16)
    got = behind(lambda s: mla.dcp_local_metadata(lens, idx, slots, 1, 2, max_pages=16, stream=s), [512])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("what", ["fork", "alloc", "compact"])
def test_page_operations(what):
    host = list(state(12, [300, 100, 640, 64, 129], 5000, 144, 53, width=40))
    if what == "compact":
        po.free(*host[1:], np.array([0, 100, 200, 0, 129] + [0] * 7))
    kv, table, lens, counts = (torch.from_numpy(x.copy()).cuda() for x in host)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = mla.pages_workspace_size(5000)
    pool = kv.view(torch.uint8).view(5000, 64, 576)
    parents, children = np.array([0, 2, 4, 1]), np.array([6, 7, 9, 11])
    new = np.array([301, 700, 640, 65, 2000] + [64] * 7)
    dp, dc, dn = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (parents, children, new))
    run = {
        "fork": lambda x, s, e: mla.pages_fork(*x, dp, dc, error_word=e, stream=s),
        "alloc": lambda x, s, e: mla.pages_alloc(*x[1:], dn, error_word=e, stream=s),
        "compact": lambda x, s, e: mla.pages_compact(x[0], x[1], x[3], error_word=e, stream=s),
    }[what]
    x = [pool, table, lens, counts]
    clones = [t.clone() for t in x]
    behind(lambda s: run(x, s, err), [n], warm=lambda s: run(clones, s, None))
    want = {"fork": lambda: po.fork(*host, parents, children), "alloc": lambda: po.alloc(*host[1:], new),
            "compact": lambda: po.compact(host[0], host[1], host[3])[0]}[what]()
    for got, h in zip((kv, table, lens, counts), host):
        np.testing.assert_array_equal(got.cpu().numpy(), h)
    assert int(err.item()) == want
    check_books(host[1], host[3])
