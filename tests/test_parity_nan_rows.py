"""A query that is not finite gives NaN in both out and lse, whether one CTA
holds its row or the schedule cut it; rows that see nothing keep the neutral
pair, and the other rows their bits."""
import math

import pytest
import torch

import mla_paged_decode_gb300 as mla
from view_cases import SCALE, buffers, causal_seen, make, run_shared, run_window, window_seen

pytestmark = pytest.mark.gpu
WIDE = 2200     # block-table columns that send 128 rows and more to the pair kernel


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


def poison(c, bad, rows):
    """Puts `bad` into one element of the given (request, head) rows of q; returns
    the mask of the other rows."""
    rest = torch.ones(c.q.shape[:3], dtype=torch.bool)
    for b, h in rows:
        c.q[b, 0, h, 100] = bad
        rest[b, 0, h] = False
    return rest


def check(good, got, rest):
    for x, y in zip(good, got):
        assert torch.equal(x[rest], y[rest])
        assert torch.isnan(y[~rest]).all()


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("base", [0, 1])
@pytest.mark.parametrize("width,heads", [(0, 16), (WIDE, 64), (WIDE, 128)])
def test_shared(kv_dtype, bad, base, width, heads):
    c = make([700, 640, 655, 0], heads, 1, kv_dtype, causal_seen(1), seed=60, shared=([0, 4], [9]), width=width)
    good = run_shared(c, [0, 4], [9], base)
    rest = poison(c, bad, [(0, 3), (1, heads - 1), (2, 0)])
    c.q[3] = bad                            # a request of length 0
    check(good, run_shared(c, [0, 4], [9], base), rest)


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("heads,copies", [(16, 1), (128, 1), (64, 60), (128, 60)])
def test_window(kv_dtype, bad, heads, copies):
    """One request of 2,000 tokens, cut across CTAs, and many that are not."""
    c = make([2000, 64, 0] * copies, heads, 1, kv_dtype, window_seen(1900, 4, 1), seed=61)
    good = run_window(c, 1900, 4)
    rest = poison(c, bad, [(b, h) for b in (0, 1) for h in (0, 5, heads - 1)])
    c.q[2] = bad
    check(good, run_window(c, 1900, 4), rest)


@pytest.mark.parametrize("num_parts", [1, 2, 3])
@pytest.mark.parametrize("length", [40000, 100])
def test_decode_partial(num_parts, length):
    """bf16: the same rule in the decode's own merge (40,000 tokens are cut)."""
    c = make([length, 64], 16, 1, "bf16", causal_seen(1), seed=62)
    ws = mla.make_workspace(c.q, c.kv, c.table)

    def run():
        out, lse = buffers(c)
        mla.decode_partial(c.q, c.kv, c.table, c.lens, 0, num_parts, SCALE, 0, out, lse, workspace=ws)
        return out, lse
    good = run()
    rest = poison(c, math.nan, [(0, 2), (1, 15)])
    check(good, run(), rest)
