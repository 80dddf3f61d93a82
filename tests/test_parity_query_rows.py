"""Queries of one call whose magnitudes differ: each request, and each row, is
held to the definition with its own largest |q|, and what one row's query holds
changes no bit of another row's result.  (Blocks of shared pages take rows of
several requests; an e4m3 cache multiplies q as two scaled fp8 terms.)"""
import math

import pytest
import torch

import mla_paged_decode_gb300 as mla
from view_cases import ViewCase, causal_seen, check, make, run_shared, run_window, window_seen

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


def check_rows(c, out, lse, requests, heads=None, what=""):
    """check, with the limits that each row's own query gives."""
    for b in requests:
        for h in heads if heads is not None else range(c.q.shape[2]):
            one = ViewCase(c.q[b:b + 1, :, h:h + 1], c.kv, c.kv_scale, c.table[b:b + 1], c.lens[b:b + 1],
                           c.seen[b:b + 1])
            check(one, out[b:b + 1, :, h:h + 1], lse[b:b + 1, :, h:h + 1], what=f"{what} request {b} head {h}")


@pytest.mark.parametrize("kv_dtype,width", KINDS)
@pytest.mark.parametrize("heads,q_len", [(16, 1), (20, 2)])
def test_requests_of_one_block_keep_their_precision(kv_dtype, width, heads, q_len):
    """Requests of scales 1, 2^12, 2^20, 2^-12 and one whose q is huge and whose
    length is 0, side by side in one group."""
    lens = [700, 655, 0, 640, 690, 641, 700, 650, 660, 671]
    gains = [0, 12, 100, 20, 0, -12, 0, 0, 20, 0]
    c = make(lens, heads, q_len, kv_dtype, causal_seen(q_len), seed=40, shared=([0, 10], [9]), width=width)
    for b, k in enumerate(gains):
        c.q[b] *= 2.0**k
    out, lse = run_shared(c, [0, 10], [9])
    check_rows(c, out, lse, range(10), heads=[0, 1, heads - 1], what="gains")


@pytest.mark.parametrize("kv_dtype,width", KINDS)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 2.0**100])
def test_a_request_changes_no_bit_of_its_neighbours(kv_dtype, width, bad):
    c = make([700, 640, 655, 0, 610, 800, 641, 666], 16, 1, kv_dtype, causal_seen(1), seed=41, shared=([0, 8], [9]),
             width=width)
    c.q[4] *= 2.0**9                      # past e4m3's largest number, unscaled
    c.q[5] *= 2.0**-9
    good, glse = run_shared(c, [0, 8], [9])
    check_rows(c, good, glse, [0, 4, 5], heads=[0, 15], what="finite")
    c.q[1, 0, 7, 3] = bad
    c.q[2, 0, 15, 570] = bad
    c.q[3] = bad                          # a request of length 0
    out, lse = run_shared(c, [0, 8], [9])
    rest = torch.ones(8, 1, 16, dtype=torch.bool)
    rest[1, 0, 7] = rest[2, 0, 15] = False
    assert torch.equal(out[rest], good[rest]) and torch.equal(lse[rest], glse[rest])
    if not math.isfinite(bad):
        assert torch.isnan(out[~rest]).all()


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,copies", [(40, 1), (128, 32)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, 2.0**100])
def test_a_row_of_a_window_changes_no_bit_of_the_others(kv_dtype, heads, copies, bad):
    """Blocks of 64 rows and (128 heads x 32 requests x 4) pairs."""
    lens = [700, 64, 0, 201] * copies
    c = make(lens, heads, 1, kv_dtype, window_seen(300, 70, 1), seed=42)
    c.q[:, :, 5] *= 2.0**9
    c.q[:, :, 6] *= 2.0**-9
    good, glse = run_window(c, 300, 70)
    check_rows(c, good, glse, [0, 1, 3], heads=[0, 5, 6, heads - 1], what="finite")
    rest = torch.ones(len(lens), 1, heads, dtype=torch.bool)
    for b, h in ((0, 7), (1, heads - 1), (3, 0)):
        c.q[b, 0, h, 575] = bad
        rest[b, 0, h] = False
    c.q[2, 0, 3] = bad                    # sees nothing: the neutral pair all the same
    out, lse = run_window(c, 300, 70)
    assert torch.equal(out[rest], good[rest]) and torch.equal(lse[rest], glse[rest])
    if not math.isfinite(bad):
        assert torch.isnan(out[~rest]).all()
