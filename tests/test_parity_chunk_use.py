"""The chunk operators as a serving loop uses them: one after the other over one
cache, captured into graphs, on streams other than the current one, from two
threads, with padded batches and bad inputs, and the same bits again."""
import math
import threading

import pytest
import torch

import chunk_cases
import expanded_cases
import mla_paged_decode_gb300 as mla
from chunk_cases import SCALE, buffers, check_attention, ints, starts_of
from test_default_scratch_streams import behind

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_written_read_and_attended(kv_dtype):
    """Chunk after chunk: each is written, attended over the cache, and what is
    read back attends to the same in two parts that are merged."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    heads, B, pages = 16, 3, 40
    scale = 5.5 / 448 if kv_dtype == "e4m3" else 1.0
    kv = torch.full((pages, 64, 576), 0x7F, dtype=torch.uint8, device="cuda") if kv_dtype == "e4m3" else \
        torch.full((pages, 64, 576), math.nan, dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(2))[:B * 12].to(torch.int32).view(B, 12).cuda()
    lens, err = [0] * B, torch.zeros(1, dtype=torch.int32, device="cuda")
    up = rnd(heads * 256, 512) / 23
    ws = mla.make_prefill_workspace(kv)
    for new in ([70, 1, 300], [130, 64, 0], [1, 200, 33]):
        starts, before = ints(starts_of(new)), ints(lens)
        x = rnd(sum(new), 576)
        mla.kv_append_chunk(x, kv, table, starts, before, kv_scale=scale, error_word=err)
        ctx_starts = ints(starts_of(lens))
        context = torch.empty(sum(lens), 576, dtype=torch.bfloat16, device="cuda")
        mla.kv_read(kv, table, ctx_starts, torch.zeros_like(before), context, kv_scale=scale, error_word=err)
        own = torch.empty_like(x)
        mla.kv_read(kv, table, starts, before, own, kv_scale=scale, error_word=err)
        if kv_dtype == "bf16":
            assert torch.equal(own, x)
        grown = [a + n for a, n in zip(lens, new)]
        c = chunk_cases.ChunkCase(rnd(sum(new), heads, 576), kv, scale, table, ints(grown), starts)
        chunk_cases.check(c, *chunk_cases.run(c, ws=ws), what=f"absorbed {new}")
        # expanded: own part and context, merged by lse
        q = rnd(sum(new), heads, 192)
        parts, lses = torch.empty(2, *q.shape[:2], 128, dtype=torch.bfloat16, device="cuda"), \
            torch.empty(2, *q.shape[:2], device="cuda")
        ups = []
        for i, (r, s) in enumerate([(own, starts), (context, ctx_starts)]):
            e = (r[:, :512] @ up.T).view(-1, heads, 256)
            ups.append(e)
            mla.prefill_expanded(q, e[..., :128], r[:, 512:], e[..., 128:], starts, s, i == 0, SCALE, 0, parts[i], lses[i],
                                 workspace=ws)
        out, lse = torch.empty_like(parts[0]), torch.empty_like(lses[0])
        mla.lse_combine(parts, lses, 2, out, out_lse=lse)
        for b, n in enumerate(new):
            if not n:
                continue
            a, k0 = sum(new[:b]), sum(lens[:b])
            e = torch.cat([ups[1][k0:k0 + lens[b]], ups[0][a:a + n]])
            rope = torch.cat([context[k0:k0 + lens[b]], own[a:a + n]])[:, None, 512:].expand(-1, heads, 64)
            k, v = torch.cat([e[..., :128], rope], -1).double(), e[..., 128:].double()
            s = torch.einsum("nhk,mhk->nhm", q[a:a + n].double(), k) * SCALE
            hide = torch.arange(grown[b], device="cuda") > lens[b] + torch.arange(n, device="cuda")[:, None]
            s = s.masked_fill(hide[:, None], -math.inf)
            want = torch.einsum("nhm,mhk->nhk", torch.softmax(s, -1), v)
            mag = torch.einsum("nhm,mhk->nhk", torch.softmax(s, -1), v.abs())
            # weights and, twice, outputs rounded to bf16 (2^-8 each), and the weights' sum
            assert ((out[a:a + n].double() - want).abs() <= 4 * 2.0**-8 * mag + 2.0**-17).all()
            assert ((lse[a:a + n].double() - torch.logsumexp(s, -1)).abs() <= 1e-4).all()
        lens = grown
    assert int(err) == 0 and mla.check_workspace(ws) == 0


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_a_graph_follows_its_batch(kv_dtype):
    """Captured once at the padded size: other lengths and starts on replay, two
    graphs on one workspace."""
    lens, news = [700, 300, 64, 129, 0], [128, 1, 64, 2, 0]
    c = chunk_cases.make(lens, news, 16, kv_dtype, seed=20, pad=60)
    e = expanded_cases.make([130, 1, 300], [200, 40, 333], 3, True, seed=21, pad=40)
    out, lse = buffers(c.q)
    eout, else_ = buffers(e.q, 128)
    rows = torch.randn(c.q.shape[0], 576, device="cuda").to(torch.bfloat16)
    back = torch.full_like(rows, 7.0)
    pos = ints([L - n for L, n in zip(lens, news)])
    keep = c.kv.clone()
    ws = mla.make_prefill_workspace(c.q)

    def step(one, two):
        if one:
            mla.kv_append_chunk(rows, c.kv, c.table, c.starts, pos, kv_scale=c.kv_scale)
            mla.kv_read(c.kv, c.table, c.starts, pos, back, kv_scale=c.kv_scale)
            mla.prefill_chunk(c.q, c.kv, c.table, c.lens, c.starts, SCALE, 0, out, lse, kv_scale=c.kv_scale, workspace=ws)
        if two:
            mla.prefill_expanded(*e.args, SCALE, 0, eout, else_, workspace=ws)
    step(True, True)
    graphs = []
    for one in (True, False):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(one, not one)
        graphs.append(g)
    for news2, shift in ((news, 0), ([60, 3, 64, 0, 0], 5), ([1, 0, 0, 129, 0], 0), ([0, 0, 0, 0, 0], 3)):
        c.kv.copy_(keep)
        c.starts.copy_(ints(starts_of(news2, shift)))
        c.lens.copy_(ints(lens))
        pos.copy_(ints([L - n for L, n in zip(lens, news2)]))
        e.q_starts.copy_(ints(starts_of([130, 1, 299 - shift], 1 + shift)))
        for t in (out, lse, eout, else_, back):
            t.fill_(7)
        for g in graphs + graphs[:1]:
            g.replay()
        chunk_cases.check(c, out, lse, what=f"replay {news2}")
        expanded_cases.check(e, eout, else_, what=f"replay {shift}")
        used = slice(shift, shift + sum(news2))
        if kv_dtype == "bf16":
            assert torch.equal(back[used], rows[used])
        assert (back[:shift] == 7).all() and (back[shift + sum(news2):] == 7).all()
    assert mla.check_workspace(ws) == 0


def test_streams_that_are_behind():
    c = chunk_cases.make([900, 64, 30], [200, 64, 1], 16, "bf16", seed=22)
    out, lse = buffers(c.q)
    n = mla.make_prefill_workspace(c.q).numel()
    behind(lambda s: mla.prefill_chunk(c.q, c.kv, c.table, c.lens, c.starts, SCALE, 0, out, lse, stream=s), [n])
    chunk_cases.check(c, out, lse)
    e = expanded_cases.make([300, 70], [900, 70], 16, True, seed=23)
    out, lse = buffers(e.q, 128)
    behind(lambda s: mla.prefill_expanded(*e.args, SCALE, 0, out, lse, stream=s), [n])
    expanded_cases.check(e, out, lse)


def test_two_threads():
    """Calls at once, each on its own stream and workspace."""
    c = chunk_cases.make([900, 64, 30], [200, 64, 1], 16, "bf16", seed=24)
    e = expanded_cases.make([600, 70], [900, 70], 16, True, seed=25)
    results, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()

    def work(case, mod, s):
        with torch.cuda.stream(s):
            ws = mla.make_prefill_workspace(case.q)
            for _ in range(20):
                r = mod.run(case, ws=ws)
            results.append((case, mod, r))
    threads = [threading.Thread(target=work, args=(x, m, s)) for (x, m), s in
               zip(((c, chunk_cases), (e, expanded_cases)), streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(results) == 2
    for case, mod, r in results:
        mod.check(case, *r)


def test_the_same_bits_again():
    c = chunk_cases.make([3000, 64, 900], [100, 64, 3], 16, "e4m3", seed=26)
    e = expanded_cases.make([600, 70, 1], [3000, 70, 900], 5, True, seed=27)
    for case, mod in ((c, chunk_cases), (e, expanded_cases)):
        a, b = mod.run(case), mod.run(case)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_batches_padded_with_empty_requests():
    news = [0] * 300 + [129, 0, 0, 3] + [0] * 200 + [70]
    lens = [0] * 300 + [400, 5, 0, 3] + [0] * 200 + [70]
    c = chunk_cases.make(lens, news, 16, "bf16", seed=28, pad=9)
    chunk_cases.check(c, *chunk_cases.run(c), what="chunk")
    for causal in (True, False):
        e = expanded_cases.make(news, lens, 16, causal, seed=29, pad=9)
        expanded_cases.check(e, *expanded_cases.run(e), what="expanded")


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_bad_entries_are_reported(kv_dtype):
    """A page or a length that is out of range spoils its own request only."""
    c = chunk_cases.make([300, 200, 100], [40, 30, 20], 16, kv_dtype, seed=30)
    ws = mla.make_prefill_workspace(c.q)
    out, lse = buffers(c.q)

    def call():
        out.fill_(7)
        lse.fill_(7)
        mla.prefill_chunk(c.q, c.kv, c.table, c.lens, c.starts, SCALE, 0, out, lse, kv_scale=c.kv_scale, workspace=ws)
    good = c.table.clone()
    for bad in (-1, c.kv.shape[0], 2**31 - 1):
        c.table[1, 2] = bad
        call()
        assert mla.check_workspace(ws) == -9
    c.table.copy_(good)
    for bad in (-5, c.table.shape[1] * 64 + 1, 2**31 - 1):
        c.lens[1] = bad
        call()
        assert mla.check_workspace(ws) == -9
    c.lens[1] = 200
    call()
    assert mla.check_workspace(ws) == 0
    chunk_cases.check(c, out, lse)


@pytest.mark.parametrize("starts", [[0, 30, 10, 50], [-7, 10, 20, 30], [0, 10, 20, 2**31 - 1], [60, 40, 20, 0]])
def test_bad_starts_stay_inside(starts):
    """Starts that fall or leave the tensors: reported, nothing outside touched."""
    c = chunk_cases.make([300, 200, 100], [40, 30, 20], 16, "bf16", seed=31)
    e = expanded_cases.make([40, 30, 20], [300, 200, 100], 4, True, seed=32)
    ws = mla.make_prefill_workspace(c.q)
    big = torch.full((c.q.shape[0] + 2, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = big[1:-1], torch.empty(c.q.shape[:2], device="cuda")
    mla.prefill_chunk(c.q, c.kv, c.table, c.lens, ints(starts), SCALE, 0, out, lse, workspace=ws)
    assert mla.check_workspace(ws) == -9
    assert (big[0] == 7).all() and (big[-1] == 7).all()
    q, kn, kr, v, qs, ks, causal = e.args
    out, lse = buffers(e.q, 128)
    for a, b in ((ints(starts), ks), (qs, ints(starts)), (ints(starts), ints(starts))):
        mla.prefill_expanded(q, kn, kr, v, a, b, causal, SCALE, 0, out, lse, workspace=ws)
        assert mla.check_workspace(ws) == -9


def test_decode_sized_chunks_agree_with_the_decode():
    """Two tokens of every request: the causal decode's result, to the roundings."""
    c = chunk_cases.make([700, 65, 128], [2, 2, 2], 64, "bf16", seed=33)
    out, lse = chunk_cases.run(c)
    o2 = torch.empty(3, 2, 64, 512, dtype=torch.bfloat16, device="cuda")
    l2 = torch.empty(3, 2, 64, device="cuda")
    mla.decode_partial(c.q.view(3, 2, 64, 576), c.kv, c.table, c.lens, 0, 1, SCALE, 0, o2, l2)
    chunk_cases.check(c, out, lse)
    assert (out.view_as(o2).float() - o2.float()).abs().max() <= 2e-2 and (lse.view_as(l2) - l2).abs().max() <= 5e-3


def test_rows_of_a_long_cache():
    """Pages past 4 GiB of the pool."""
    pages = 60000
    kv = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    c = chunk_cases.make([500], [70], 16, "bf16", seed=34)
    far = ints([[pages - 1 - 3 * i for i in range(8)]])
    kv[far[0].long()] = c.kv[c.table[0].long()]
    c.kv, c.table = kv, far
    chunk_cases.check(c, *chunk_cases.run(c), what="far")


def test_large_heads_and_queries_offsets():
    """Outputs past 2^31 values."""
    n = 40000
    c = chunk_cases.make([300], [300], 128, "bf16", seed=35)
    q = torch.zeros(n, 128, 576, dtype=torch.bfloat16, device="cuda")
    q[n - 300:] = c.q
    out, lse = torch.zeros(n, 128, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 128, device="cuda")
    mla.prefill_chunk(q, c.kv, c.table, c.lens, ints([n - 300, n]), SCALE, 0, out, lse)
    assert out.numel() > 2**31 and not out[:n - 300].any()
    tail_out, tail_lse = buffers(c.q)
    tail_out.copy_(out[n - 300:])
    tail_lse.copy_(lse[n - 300:])
    chunk_cases.check(c, tail_out, tail_lse, what="tail")


def test_check_attention_notices():
    """The checks themselves: a value off by its limit's size is noticed."""
    c = chunk_cases.make([100], [10], 2, "bf16", seed=36)
    out, lse = chunk_cases.run(c)
    out[3, 1, 5] += 0.25
    with pytest.raises(AssertionError):
        chunk_cases.check(c, out, lse)
    assert check_attention is chunk_cases.check_attention
