"""Views at the ends of their ranges: block tables of 2^25 columns and more, and
requests of up to 2^31 - 64 tokens (whose pages repeat in the table)."""

import pytest
import torch

import mla_paged_decode_gb300 as mla
from view_cases import SCALE, ViewCase, buffers, causal_seen, check, make, run_shared, run_window, window_seen

pytestmark = pytest.mark.gpu
TOP = 2**31 - 64


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


def widen(c, width):
    wide = torch.full((c.table.shape[0], width), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide


@pytest.mark.parametrize("width", [2**25 - 1, 2**25, 2**25 + 1])
@pytest.mark.parametrize("heads", [16, 128])
def test_tables_as_wide_as_lengths_go(width, heads):
    c = make([300, 0], heads, 1, "e4m3", window_seen(100, 5, 1), seed=90)
    widen(c, width)
    check(c, *run_window(c, 100, 5), what="window")
    c = make([300, 260], heads, 1, "bf16", causal_seen(1), seed=91, shared=([0, 2], [4]))
    widen(c, width)
    check(c, *run_shared(c, [0, 2], [4]), what="shared")
    out, lse = buffers(c)
    ws = mla.make_workspace(c.q, c.kv, c.table)
    mla.decode_partial(c.q, c.kv, c.table, c.lens, 0, 1, SCALE, 0, out, lse, workspace=ws)
    assert mla.check_workspace(ws) == 0
    want = run_shared(c, [0, 2], [4])[0]
    assert (out.float() - want.float()).abs().max() <= 2.0**-6 * want.float().abs().max()


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,q_len", [(16, 1), (64, 2), (128, 3)])
@pytest.mark.parametrize("length,window,sinks", [(TOP, 100, 5), (TOP - 1, 300, 0), (TOP, 700, 70), (TOP - 250, 64, 1)])
def test_windows_at_the_end_of_the_longest_request(kv_dtype, heads, q_len, length, window, sinks):
    """Only the sinks' and the window's pages are in the table; the rows that no
    query sees hold NaN."""
    near = 1024 + length % 64                   # the same request, moved down by whole pages
    c = make([near], heads, q_len, kv_dtype, window_seen(window, sinks, q_len), seed=92)
    first = (length - near) // 64
    table = torch.full((1, 2**25), -1, dtype=torch.int32, device="cuda")
    used = c.table.shape[1]
    keep = min(-(-sinks // 64), used)
    table[0, first:first + used] = c.table[0]
    if first:
        table[0, first:first + keep] = -1
    table[0, :keep] = c.table[0, :keep]
    far = ViewCase(c.q, c.kv, c.kv_scale, table, torch.tensor([length], dtype=torch.int32, device="cuda"), c.seen)
    out, lse = run_window(far, window, sinks)
    check(c, out, lse, what=f"length {length}")


@pytest.mark.parametrize("heads", [16, 128])
def test_lengths_past_the_longest_are_reported(heads):
    c = make([300], heads, 1, "e4m3", window_seen(100, 0, 1), seed=93)
    widen(c, 2**25)
    c.table[0, -5:] = 0
    c.lens[0] = 2**31 - 1
    out, lse = buffers(c)
    ws = mla.make_workspace(c.q, c.kv, c.table, c.kv_scale)
    mla.decode_window(c.q, c.kv, c.table, c.lens, 100, 0, SCALE, 0, out, lse, kv_scale=c.kv_scale, workspace=ws)
    assert mla.check_workspace(ws) == -9
