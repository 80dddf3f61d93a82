"""The combine of partitions whose lse is NaN is NaN, also when all of them are
(a NaN query): only a row of nothing but -inf is the neutral pair."""
import math

import pytest
import torch

import mla_paged_decode_gb300 as mla
from view_cases import SCALE, causal_seen, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


@pytest.mark.parametrize("parts,dim", [(1, 512), (2, 512), (8, 512), (33, 512), (100, 64), (3, 1024)])
def test_lse_combine(parts, dim):
    g = torch.Generator(device="cuda").manual_seed(parts)
    x = torch.randn(parts, 5, 3, dim, generator=g, device="cuda").to(torch.bfloat16)
    lses = torch.randn(parts, 5, 3, generator=g, device="cuda")
    lses[:, 1] = -math.inf
    good, glse = torch.empty(5, 3, dim, dtype=torch.bfloat16, device="cuda"), torch.empty(5, 3, device="cuda")
    mla.lse_combine(x, lses, parts, good, out_lse=glse)
    lses[:, 0, 1] = math.nan                # all of a row
    lses[parts - 1, 2, 2] = math.nan        # one of a row
    lses[0, 3, 0] = math.nan
    lses[1:, 3, 0] = -math.inf              # the others own nothing
    out, lse = torch.empty_like(good), torch.empty_like(glse)
    mla.lse_combine(x, lses, parts, out, out_lse=lse)
    rest = torch.ones(5, 3, dtype=torch.bool)
    for t, h in ((0, 1), (2, 2), (3, 0)):
        rest[t, h] = False
    assert torch.isnan(out[~rest]).all() and torch.isnan(lse[~rest]).all()
    assert torch.equal(out[rest], good[rest]) and torch.equal(lse[rest], glse[rest])
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("num_parts", [2, 3, 8, 9])
def test_decode_dcp(num_parts):
    c = make([9000, 100, 0], 16, 1, "bf16", causal_seen(1), seed=63)
    glse, lse = torch.empty(3, 1, 16, device="cuda"), torch.empty(3, 1, 16, device="cuda")
    good = mla.decode_dcp(c.q, c.kv, c.table, c.lens, num_parts, SCALE, 0, out_lse=glse)[0]
    c.q[0, 0, 3, 9] = math.nan
    c.q[1, 0, 15, 570] = math.nan
    c.q[2] = math.nan                       # sees nothing
    out = mla.decode_dcp(c.q, c.kv, c.table, c.lens, num_parts, SCALE, 0, out_lse=lse)[0]
    rest = torch.ones(3, 1, 16, dtype=torch.bool)
    rest[0, 0, 3] = rest[1, 0, 15] = False
    assert torch.isnan(out[~rest]).all() and torch.isnan(lse[~rest]).all()
    assert torch.equal(out[rest], good[rest]) and torch.equal(lse[rest], glse[rest])
