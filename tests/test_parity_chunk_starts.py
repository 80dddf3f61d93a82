"""Starts of kv_append_chunk and kv_read that fall or leave the buffer are
reported, and touch nothing but rows of the buffer and of the requests' pages."""
import pytest
import torch

import mla_paged_decode_gb300 as mla
from chunk_cases import ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


BAD = [[0, 30, 10], [-5, 10, 20], [10, 10**9, 2**31 - 1], [0, 10, 41], [30, 20, 10], [0, 0, -1], [-2**31, 0, 40],
       [0, 2**31 - 1, 40]]


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("starts", BAD)
def test_bad_starts_are_reported_and_stay_inside(kv_dtype, starts):
    g = torch.Generator().manual_seed(1)
    n, margin, pages = 40, 8, 4
    around = torch.randint(0, 127, (pages + 2, 64, 576 * (1 if kv_dtype == "e4m3" else 2)), generator=g,
                           dtype=torch.uint8).cuda()
    pool = around[1:-1] if kv_dtype == "e4m3" else around[1:-1].view(torch.bfloat16)
    table, pos = ints([[2], [0]]), ints([0, 3])     # pages 1 and 3 are nobody's
    rows = torch.randn(n + 2 * margin, 576, generator=g).to(torch.bfloat16).cuda()
    before, err = around.clone(), word()
    mla.kv_append_chunk(rows[margin:-margin], pool, table, ints(starts), pos, error_word=err)
    assert int(err) & 2
    for page in (0, 2, 4, 5):                       # the margins and the pages of nobody
        assert torch.equal(around[page], before[page])

    wide = torch.full((n + 2 * margin, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    err.zero_()
    mla.kv_read(pool, table, ints(starts), pos, wide[margin:-margin], error_word=err)
    assert int(err) & 2
    assert (wide[:margin] == 5).all() and (wide[-margin:] == 5).all()
    held = pool.view(torch.float8_e4m3fn).float() if kv_dtype == "e4m3" else pool.float()
    held = torch.cat([held[2], held[0], torch.zeros(1, 576, device="cuda"), torch.full((1, 576), 5.0, device="cuda")])
    got = wide[margin:-margin].float()
    assert (got[:, None] == held).all(-1).any(-1).all()   # a row of the requests' pages, zeros, or as it was


@pytest.mark.parametrize("starts,positions,code", [([0, 10, 40], [0, 3], 0), ([3, 3, 17], [0, 0], 0),
                                                   ([40, 40, 40], [0, 0], 0), ([0, 20, 40], [100, 0], 1),
                                                   ([0, 20, 19], [100, 0], 3)])
def test_good_starts_and_missing_pages(starts, positions, code):
    """Bit 1 for starts alone, bit 0 for pages alone."""
    pool = torch.zeros(4, 64, 576, dtype=torch.bfloat16, device="cuda")
    rows, table, err = torch.ones(40, 576, dtype=torch.bfloat16, device="cuda"), ints([[2], [0]]), word()
    mla.kv_append_chunk(rows, pool, table, ints(starts), ints(positions), error_word=err)
    assert int(err) == code
    err.zero_()
    mla.kv_read(pool, table, ints(starts), ints(positions), rows, error_word=err)
    assert int(err) == code


@pytest.mark.parametrize("batch", [1, 128, 129, 1000])
def test_every_request_is_looked_at(batch):
    """Few rows of many requests: the last request's starts as well."""
    pool = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda")
    rows, err = torch.ones(3, 576, dtype=torch.bfloat16, device="cuda"), word()
    table, pos, starts = ints([[0]] * batch), ints([0] * batch), ints([0] * batch + [3])
    mla.kv_append_chunk(rows, pool, table, starts, pos, error_word=err)
    assert int(err) == 0 and (pool[0, :3] == 1).all() and not pool[0, 3:].any()
    starts[batch] = 4
    mla.kv_append_chunk(rows, pool, table, starts, pos, error_word=err)
    assert int(err) == 2
    err.zero_()
    mla.kv_read(pool, table, starts, pos, rows, error_word=err)
    assert int(err) == 2
