"""Ragged batches drawn at random, against the 64-bit definitions: where blocks,
tiles, ranges and requests begin and end depends on all lengths at once."""
import math
import random

import pytest
import torch

import chunk_cases
import expanded_cases

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    import mla_paged_decode_gb300 as mla
    mla.load_library()


def draw(seed):
    """Queries and tokens of each request: up to 600 requests, many of them
    empty, some with fewer tokens than queries."""
    r = random.Random(seed)
    spread = lambda a, b: int(round(math.exp(r.uniform(math.log(a), math.log(b)))))  # noqa: E731
    requests, total = spread(1, 600), spread(1, 3000)
    news = [0] * requests
    for _ in range(min(total, 400)):
        news[r.randrange(requests)] += max(1, total // 400)
    if r.random() < 0.5:
        news = [n if r.random() < 0.3 else 0 for n in news]
    tokens = [max(0, n + r.choice([0, 0, -3, spread(1, 2000) if r.random() < 0.2 else r.randrange(40)])) for n in news]
    while sum(tokens) > 60000:
        tokens[tokens.index(max(tokens))] = 1
    return r, news, tokens, r.choice([1, 2, 3, 5, 16]), r.choice([0, 5])


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_chunk(kv_dtype, seed):
    _, news, tokens, heads, pad = draw(seed)
    c = chunk_cases.make(tokens, news, heads, kv_dtype, seed, pad=pad)
    chunk_cases.check(c, *chunk_cases.run(c), what=f"seed {seed}")


@pytest.mark.parametrize("seed", range(100, 120))
def test_expanded(seed):
    r, news, tokens, heads, pad = draw(seed)
    c = expanded_cases.make(news, tokens, heads, r.random() < 0.6, seed, pad=pad)
    expanded_cases.check(c, *expanded_cases.run(c), what=f"seed {seed}")
