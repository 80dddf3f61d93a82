"""Groups of decode_shared whose requests end or are shorter than the shared
pages: the others keep their results whichever request that is."""
import math

import pytest
import torch

import mla_paged_decode_gb300 as mla
from view_cases import SCALE, buffers, causal_seen, check, make, run_shared

pytestmark = pytest.mark.gpu
WIDE = 2200     # block-table columns that send 128 rows and more to the pair kernel
KINDS = [("bf16", 0), ("bf16", WIDE), ("e4m3", 0), ("e4m3", WIDE)]


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


def end(c, requests):
    """The requests have ended: length 0, their rows given up."""
    for b in requests:
        c.lens[b] = 0
        c.table[b] = -1
        c.seen[b] = [torch.arange(0) for _ in c.seen[b]]


@pytest.mark.parametrize("kv_dtype,width", KINDS)
@pytest.mark.parametrize("heads,q_len", [(16, 1), (64, 1), (128, 2)])
@pytest.mark.parametrize("ended", [[0], [0, 1, 2], [3], [0, 5, 8], [0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 6, 7, 8]])
def test_requests_of_a_group_may_end(kv_dtype, width, heads, q_len, ended):
    lens = [700, 640, 655, 1001, 642, 704, 130, 160, 129]
    c = make(lens, heads, q_len, kv_dtype, causal_seen(q_len), seed=80, shared=([0, 6, 9], [10, 2]), width=width)
    end(c, ended)
    check(c, *run_shared(c, [0, 6, 9], [10, 2]), what=f"ended {ended}")


@pytest.mark.parametrize("kv_dtype,width", KINDS)
def test_short_requests_need_not_name_the_shared_pages(kv_dtype, width):
    """Each row names its own pages only; one of many reaches the shared ones."""
    lens = [(7 * b) % 600 for b in range(40)] + [777]
    c = make(lens, 16, 1, kv_dtype, causal_seen(1), seed=81, shared=([0, 41], [12]), width=width)
    for b, n in enumerate(lens):
        c.table[b, -(-n // 64):] = -1
    check(c, *run_shared(c, [0, 41], [12]), what="short")


@pytest.mark.parametrize("kv_dtype,width", KINDS)
@pytest.mark.parametrize("heads,q_len", [(64, 1), (100, 2)])
def test_no_request_reaches_the_shared_pages(kv_dtype, width, heads, q_len):
    lens = [320, 100, 0, 449, 64, 448]
    c = make(lens, heads, q_len, kv_dtype, causal_seen(q_len), seed=82, shared=([0, 6], [12]), width=width)
    for b, n in enumerate(lens):
        c.table[b, -(-n // 64):] = -1
    check(c, *run_shared(c, [0, 6], [12]), what="none reaches")


@pytest.mark.parametrize("kv_dtype,width", KINDS)
@pytest.mark.parametrize("heads,q_len", [(64, 1), (100, 2)])
@pytest.mark.parametrize("longest", [449, 257, 256, 255, 65, 1])
def test_rows_past_every_request_may_hold_anything(kv_dtype, width, heads, q_len, longest):
    """The last shared page is partly written: its other rows hold NaN."""
    lens = [min(320, longest), 0, longest, min(100, longest)]
    c = make(lens, heads, q_len, kv_dtype, causal_seen(q_len), seed=85, shared=([0, 4], [12]), width=width)
    at = torch.arange(longest, 12 * 64, device="cuda")
    if kv_dtype == "e4m3":
        c.kv[c.table[2, at // 64].long(), at % 64] = 0x7F
    else:
        c.kv[c.table[2, at // 64].long(), at % 64] = math.nan
    check(c, *run_shared(c, [0, 4], [12]), what=f"longest {longest}")


@pytest.mark.parametrize("kv_dtype,width", KINDS)
def test_all_requests_of_a_group_have_ended(kv_dtype, width):
    c = make([700, 640, 655, 300, 260], 64, 1, kv_dtype, causal_seen(1), seed=83, shared=([0, 3, 5], [10, 4]), width=width)
    end(c, [0, 1, 2])
    check(c, *run_shared(c, [0, 3, 5], [10, 4]), what="one group ended")
    end(c, [3, 4])
    check(c, *run_shared(c, [0, 3, 5], [10, 4]), what="both ended")


def test_a_bad_entry_of_the_request_that_is_read_is_reported():
    for width in (0, WIDE):
        c = make([640, 655], 128, 1, "bf16", causal_seen(1), seed=84, shared=([0, 2], [10]), width=width)
        end(c, [0])
        c.table[1, 4] = c.kv.shape[0]
        out, lse = buffers(c)
        ws = mla.make_shared_workspace(c.q, c.kv, c.table, 1)
        mla.decode_shared(c.q, c.kv, c.table, c.lens, torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
                          torch.tensor([10], dtype=torch.int32, device="cuda"), SCALE, 0, out, lse, workspace=ws)
        assert mla.check_workspace(ws) == -9
        assert (out[0] == 0).all() and (lse[0] == -math.inf).all()


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,width,shape", [(20, 0, "many groups"), (40, WIDE, "many groups"),
                                               (64, WIDE, "one group"), (128, WIDE, "one group"),
                                               (16, 0, "one group")])
def test_ended_and_short_requests_among_hundreds(kv_dtype, heads, width, shape):
    """More requests than threads: the schedule walks them in chunks, before and
    after the groups' readers are looked up."""
    g = torch.Generator().manual_seed(heads)
    if shape == "many groups":
        starts, pages = [0], []
        for k in range(90):
            starts.append(starts[-1] + (k * 7) % 9)
            pages.append((k * 5) % 7)
    else:
        starts, pages = [0, 410], [6]
    lens, full = [], []
    for k, n in enumerate(pages):
        for _ in range(starts[k], starts[k + 1]):
            full.append(64 * n + int(torch.randint(1, 150, (), generator=g)))
            r = float(torch.rand((), generator=g))
            # ended, shorter than the shared pages, or neither; one group in three has nobody at full length
            lens.append(0 if r < 0.5 else full[-1] if r > 0.7 and k % 3 else int(full[-1] * (r - 0.4)))
    c = make(full, heads, 1, kv_dtype, causal_seen(1), seed=86, shared=(starts, pages), width=width)
    for b, n in enumerate(lens):
        c.table[b, -(-n // 64):] = -1
    c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    c.seen = [[torch.arange(n)] for n in lens]
    check(c, *run_shared(c, starts, pages), what=shape)
