"""GPU parity of prefill_expanded with its definition in 64 bits: one token to
thousands, requests without queries or keys, fewer keys than queries, blocks
and tiles cut everywhere, masks on and off."""
import math

import pytest
import torch

import mla_paged_decode_gb300 as mla
from chunk_cases import SCALE, buffers, ints
from expanded_cases import check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


BATCHES = [
    # queries, keys
    ([1], [1]),
    ([200], [200]),
    ([128, 256, 512], [128, 256, 512]),
    ([127, 257, 513, 129], [129, 300, 1000, 1]),
    ([0, 5, 3, 0, 700], [9, 5, 0, 0, 900]),
    ([600, 70], [3, 129]),                        # fewer keys than queries: the first see nothing
    ([1, 1, 1, 1], [1, 127, 128, 1029]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [1, 3, 16])
@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_expanded(causal, heads, batch):
    news, keys = BATCHES[batch]
    c = make(news, keys, heads, causal, seed=heads + batch, pad=9 * (batch % 2))
    base = heads % 2
    check(c, *run(c, base), base, f"batch {batch}")


@pytest.mark.parametrize("causal", [True, False])
def test_many_heads_and_long_keys(causal):
    c = make([300, 40], [1500, 260], 128, causal, seed=3)
    check(c, *run(c), what="heads")
    c = make([1], [20000], 2, causal, seed=4)
    check(c, *run(c), what="one query")
    c = make([2000], [5000], 2, causal, seed=5)
    check(c, *run(c), what="long")
    n = [(37 * b) % 90 for b in range(410)]
    c = make(n, [x + b % 50 for b, x in enumerate(n)], 2, causal, seed=6)
    check(c, *run(c), what="many")


@pytest.mark.parametrize("gain", [0.0, 60.0])
def test_flat_and_steep_scores(gain):
    c = make([300, 90], [700, 90], 4, True, seed=9, q_gain=gain)
    check(c, *run(c), what=f"gain {gain}")


def test_offsets_of_the_first_starts():
    c = make([7, 150, 20], [11, 260, 30], 4, True, seed=10, pad=50)
    c.q_starts, c.k_starts = c.q_starts[1:].contiguous(), c.k_starts[1:].contiguous()  # the first is nobody's
    check(c, *run(c), what="offset")


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_another_requests_rows_stay_its_own(bad):
    c = make([100, 60, 300], [140, 65, 333], 4, True, seed=11)
    first, end = int(c.k_starts[1]), int(c.k_starts[2])
    c.up[first:end] = bad
    c.latent[first:end] = bad
    out, lse = buffers(c.q, 128)
    mla.prefill_expanded(*c.args, SCALE, 0, out, lse)
    a, b = int(c.q_starts[1]), int(c.q_starts[2])
    assert torch.isnan(out[a:b].float()).all()
    out[a:b], lse[a:b] = 0, 0
    check(c, out, lse, what="others", skip=(1,))


def test_contiguous_tensors_and_no_keys():
    c = make([70], [130], 3, True, seed=12)
    out, lse = run(c)
    o2, l2 = buffers(c.q, 128)
    q, kn, kr, v, *rest = c.args
    mla.prefill_expanded(q, kn.contiguous(), kr.contiguous(), v.contiguous(), *rest, SCALE, 0, o2, l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    empty = torch.empty(0, 3, 128, dtype=torch.bfloat16, device="cuda")
    mla.prefill_expanded(q, empty, torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), empty, c.q_starts,
                         ints([0, 0]), False, SCALE, 0, o2, l2)
    assert (o2 == 0).all() and torch.isneginf(l2).all()
