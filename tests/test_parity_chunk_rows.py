"""GPU parity of kv_append_chunk and kv_read with their definition: ragged
batches, both cache types, partitions, rows inside wider ones, rows of nobody,
pages that are missing."""
import math

import pytest
import torch

import mla_paged_decode_gb300 as mla
from chunk_cases import ints, starts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


def setup(news, positions, kv_dtype, seed, first=0, pad=0, wide=0):
    g = torch.Generator().manual_seed(seed)
    need = [-(-(max(p, 0) + n) // 64) for n, p in zip(news, positions)]
    total = sum(need) + 2
    perm = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(news), max(1, max(need, default=1))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    n = first + sum(news) + pad
    rows = (torch.randn(n, 576 + wide, generator=g) * 3).to(torch.bfloat16)
    if n:
        rows[0, :8] = torch.tensor([0.0, -0.0, 1e4, -1e4, math.inf, -math.inf, math.nan, 2.0**-30])
    kv = torch.randint(0, 255, (total, 64, 576 * (1 if kv_dtype == "e4m3" else 2)), generator=g, dtype=torch.uint8)
    kv = kv.cuda() if kv_dtype == "e4m3" else kv.cuda().view(torch.bfloat16)
    return rows.cuda()[:, :576], kv, table.cuda(), ints(starts_of(news, first)), ints(positions)


def codes(x, scale):
    """e4m3 of fp32(x) / scale: the exact division of the fp32 values (a quotient of
    two fp32 numbers that is rounded to fp64 and then to fp32 is rounded right)."""
    y = (x.double() / scale).float()
    c = y.clamp(-448, 448).to(torch.float8_e4m3fn)
    return torch.where(torch.isnan(y), torch.tensor(math.nan), c.float()).to(torch.float8_e4m3fn).view(torch.uint8)


def expected(rows, kv, table, starts, positions, scale, part=0, parts=1):
    want, rows, table = kv.cpu().clone(), rows.cpu(), table.cpu()
    flat = want.view(-1, 576)
    s = starts.tolist()
    for b, p in enumerate(positions.tolist()):
        if p < 0:
            continue
        t = p + torch.arange(s[b + 1] - s[b])
        own = t % parts == part
        page = torch.where(t // 64 < table.shape[1], table[b, (t // 64).clamp(max=table.shape[1] - 1)], -1)
        ok = own & (page >= 0) & (page < kv.shape[0])
        x = rows[s[b]:s[b + 1]][ok]
        flat[page[ok].long() * 64 + t[ok] % 64] = codes(x, scale) if kv.dtype == torch.uint8 else x
    return want


def same(a, b):
    """Bit for bit, any NaN for a NaN."""
    if a.dtype == torch.uint8:
        return bool(((a == b) | ((a & 0x7F == 0x7F) & (b & 0x7F == 0x7F))).all())
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


BATCHES = [
    # news, positions
    ([1], [0]),
    ([5], [62]),
    ([0, 3, 0], [0, 7, 9]),
    ([1, 64, 65, 0, 130, 7], [0, 64, 63, 5, 1, 1000]),
    ([33, 2, 9], [10, -1, 40]),
    ([1] * 70 + [200], list(range(70)) + [3]),
    ([700, 1, 999], [5000, 12, 63]),
]


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("first,pad,wide", [(0, 0, 0), (3, 10, 64), (0, 1, 8)])
@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_append_and_read(kv_dtype, first, pad, wide, batch):
    news, positions = BATCHES[batch]
    rows, kv, table, starts, pos = setup(news, positions, kv_dtype, batch, first, pad, wide)
    scale = 0.037 if kv_dtype == "e4m3" else 1.0
    want = expected(rows, kv, table, starts, pos, torch.tensor(scale).double().float().double())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert mla.kv_append_chunk(rows, kv, table, starts, pos, kv_scale=scale, error_word=err) is kv
    assert int(err) == 0 and same(kv.cpu(), want)

    wide_out = torch.full((rows.shape[0], 576 + wide), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide_out[:, :576]
    mla.kv_read(kv, table, starts, pos, out, kv_scale=scale, error_word=err)
    back = torch.full(out.shape, 5.0, dtype=torch.bfloat16)
    s = starts.tolist()
    flat = want.view(-1, 576)
    for b, p in enumerate(positions):
        if p >= 0:
            t = p + torch.arange(news[b])
            x = flat[table.cpu()[b, t // 64].long() * 64 + t % 64]
            back[s[b]:s[b + 1]] = (x.view(torch.float8_e4m3fn).float() * scale).to(torch.bfloat16) \
                if kv_dtype == "e4m3" else x
    got = out.cpu()
    nan = torch.isnan(back)
    assert int(err) == 0 and torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan].view(torch.int16), back[~nan].view(torch.int16))
    assert (wide_out[:, 576:] == 5).all()


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("parts", [2, 3, 8])
def test_append_of_a_partition(kv_dtype, parts):
    news, positions = [9, 130, 1], [5, 63, 64]
    for part in range(parts):
        rows, kv, table, starts, pos = setup(news, positions, kv_dtype, 11)
        want = expected(rows, kv, table, starts, pos, 1.0, part, parts)
        mla.kv_append_chunk(rows, kv, table, starts, pos, part, parts)
        assert same(kv.cpu(), want)


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_missing_pages(kv_dtype):
    rows, kv, table, starts, pos = setup([70, 5, 4], [60, 3, 0], kv_dtype, 3)
    pos[2] = 2**31 - 3           # tokens past 2^31: no page
    table[0, 1] = kv.shape[0]    # tokens 64 .. 127
    table[1, 0] = -1
    want = expected(rows, kv, table, starts, ints([60, 3, -1]), 1.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.kv_append_chunk(rows, kv, table, starts, pos, error_word=err)
    assert int(err) == 1 and same(kv.cpu(), want)
    mla.kv_append_chunk(rows, kv, table, starts, pos)  # without a word: skipped alike
    assert same(kv.cpu(), want)
    err.zero_()
    out = torch.full(rows.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    mla.kv_read(kv, table, starts, pos, out, error_word=err)
    page = torch.cat([(60 + torch.arange(70)) // 64, torch.full((9,), 1)])
    assert int(err) == 1 and (out.cpu()[page == 1] == 0).all()
    assert not (out.cpu()[page != 1] == 5).all()


def test_starts_out_of_range_touch_nothing_else():
    """Starts that fall, or pass the buffer: rows inside the buffer only."""
    rows, kv, table, _, pos = setup([20, 20], [0, 0], "bf16", 5)
    for bad in ([0, 30, 10], [-5, 10, 20], [10, 10**9, 2**31 - 1]):
        mla.kv_append_chunk(rows, kv, table, ints(bad), pos)
        mla.kv_read(kv, table, ints(bad), pos, torch.empty_like(rows))
    torch.cuda.synchronize()


def test_pages_past_four_gib():
    """Rows at offsets that pass 32 bits."""
    pages = 60000
    kv = torch.empty(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    table = ints([[pages - 1, 59000]])
    rows = torch.randn(100, 576, device="cuda").to(torch.bfloat16)
    mla.kv_append_chunk(rows, kv, table, ints([0, 100]), ints([20]))
    assert torch.equal(kv[pages - 1, 20:], rows[:44]) and torch.equal(kv[59000, :56], rows[44:])
    out = torch.empty_like(rows)
    mla.kv_read(kv, table, ints([0, 100]), ints([20]), out)
    assert torch.equal(out, rows)


@pytest.mark.parametrize("scale", [0.037, 5.5 / 448.0, 1.0, 2.0**-7, 3.0, 1.0 / 3.0, 1e-32, 1e32, 448.0, 0.011718751, 2.0**-30, 2.0**30,
                                   2.0 - 2.0**-23, 1.0 + 2.0**-23, 2.0**-31, 0.1, 7e-9, 0.7071068, 1.9999995e-3])
def test_every_bf16_value_is_quantised_as_the_division_says(scale):
    """All 65,536 bf16 values, over scales inside and outside the range that the
    quotient is worked out in without a division."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    rows = torch.zeros(114 * 576, dtype=torch.int16)
    rows[:65536] = bits
    rows = rows.view(torch.bfloat16).view(114, 576).cuda()
    kv = torch.zeros(2, 64, 576, dtype=torch.uint8, device="cuda")
    table, starts, pos = ints([[1, 0]]), ints([0, 114]), ints([3])
    s32 = torch.tensor(scale, dtype=torch.float32).double()
    want = expected(rows, kv, table, starts, pos, s32)
    mla.kv_append_chunk(rows, kv, table, starts, pos, kv_scale=scale)
    assert same(kv.cpu(), want)
