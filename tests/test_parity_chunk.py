"""GPU parity of prefill_chunk with its definition in 64 bits: chunks from one
token to hundreds beside one another, head counts that leave blocks part full
and put several tokens into one, requests that are empty or shorter than their
chunk, padding, both cache types, NaN in every row out of view."""
import pytest
import torch

import mla_paged_decode_gb300 as mla
from chunk_cases import check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


BATCHES = [
    # lens, news
    ([1], [1]),
    ([300], [48]),
    ([64, 65, 63, 128], [64, 1, 2, 127]),
    ([0, 5, 700, 0, 130], [0, 5, 3, 4, 129]),     # empty requests, one with queries that see nothing
    ([3, 40, 257], [9, 70, 300]),                 # fewer tokens than queries: the first see nothing
    ([1000] + [77 + 64 * k for k in range(6)], [257, 1, 1, 1, 1, 1, 1]),
]


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [1, 7, 16, 20, 64, 65, 128])
@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_chunk(kv_dtype, heads, batch):
    lens, news = BATCHES[batch]
    c = make(lens, news, heads, kv_dtype, seed=heads + batch, pad=5 * (batch % 2))
    base = heads % 2
    check(c, *run(c, base), base, f"batch {batch}")


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_long_requests_and_many(kv_dtype):
    c = make([9000, 4096, 12001], [300, 3, 70], 16, kv_dtype, seed=6, pad=3)
    check(c, *run(c), what="long")
    c = make([20000], [1], 128, kv_dtype, seed=7)
    check(c, *run(c), what="one")
    c = make([(37 * b) % 300 for b in range(410)], [min((37 * b) % 300, b % 4) for b in range(410)], 5, kv_dtype, seed=8)
    check(c, *run(c), what="many")


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("gain", [0.0, 40.0])
def test_flat_and_steep_scores(kv_dtype, gain):
    c = make([700, 90], [129, 90], 16, kv_dtype, seed=9, q_gain=gain)
    check(c, *run(c), what=f"gain {gain}")


def test_the_first_start_may_be_past_zero():
    c = make([200, 100], [30, 20], 16, "bf16", seed=10, pad=50)
    c.starts += 7
    check(c, *run(c), what="offset")
