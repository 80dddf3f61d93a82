"""GPU parity of the prefill attention over long contexts in the 2-norm, request by
request and head by head (norm_checks): a lost key, a mask off by one or weights
of fewer bits are ten times what the formats' roundings give."""
import pytest
import torch

import chunk_cases
import expanded_cases
import mla_paged_decode_gb300 as mla
from norm_checks import check_chunk, check_expanded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


CHUNKS = [  # lens, news, heads
    ([20000], [40], 2),
    ([9000, 4096, 12001], [300, 3, 70], 16),
    ([5000, 700], [64, 33], 128),
    ([2000 + 61 * b for b in range(30)], [1 + 7 * (b % 5) for b in range(30)], 16),
    ([20000], [1], 128),
    ([3000], [1000], 5),
]


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_chunk(kv_dtype, case):
    lens, news, heads = CHUNKS[case]
    c = chunk_cases.make(lens, news, heads, kv_dtype, seed=70 + case, pad=case % 3)
    base = case % 2
    check_chunk(c, *chunk_cases.run(c, base), base, f"case {case}")


EXPANDED = [  # news, keys, heads
    ([40], [5000], 2),
    ([300, 40], [1500, 1260], 128),
    ([2000], [5000], 2),
    ([256, 1, 77], [20000, 4096, 3001], 5),      # both halves on the same rows
    ([600, 513, 129, 300], [2000, 3000, 1024, 5001], 16),
    ([5 + 11 * b for b in range(25)], [900 + 83 * b for b in range(25)], 3),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(EXPANDED)))
def test_expanded(causal, case):
    news, keys, heads = EXPANDED[case]
    c = expanded_cases.make(news, keys, heads, causal, seed=80 + case, pad=case % 3)
    base = case % 2
    check_expanded(c, *expanded_cases.run(c, base), base, f"case {case}")
