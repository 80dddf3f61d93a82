"""Bad starts, pages and lengths in the prefill calls: outputs lie inside larger
buffers whose margins stay, and the requests beside a bad one get theirs."""
import pytest
import torch

import chunk_cases
import expanded_cases
import mla_paged_decode_gb300 as mla
from chunk_cases import SCALE, check_attention, ints, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


class Margins:
    """out and lse of [n, heads, dim] inside larger buffers full of sevens."""

    def __init__(self, n, heads, dim, rows=8):
        self.rows = rows
        self.out_all = torch.full((n + 2 * rows, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse_all = torch.full((n + 2 * rows, heads), 7.0, device="cuda")
        self.out, self.lse = self.out_all[rows:-rows], self.lse_all[rows:-rows]

    def kept(self):
        return all(bool((t[part] == 7).all()) for t in (self.out_all, self.lse_all)
                   for part in (slice(0, self.rows), slice(-self.rows, None)))


BAD = [[0, 30, 10, 50], [-7, 10, 20, 30], [0, 10, 20, 2**31 - 1], [60, 40, 20, 0], [0, 40, 70, 91],
       [-2**31, 2**31 - 1, -1, 2**31 - 1]]


@pytest.mark.parametrize("starts", BAD)
@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [3, 16])
def test_chunk_with_bad_starts(kv_dtype, heads, starts):
    c = chunk_cases.make([300, 200, 100], [40, 30, 20], heads, kv_dtype, seed=31)
    ws, m = mla.make_prefill_workspace(c.q), Margins(90, heads, 512)
    mla.prefill_chunk(c.q, c.kv, c.table, c.lens, ints(starts), SCALE, 0, m.out, m.lse, kv_scale=c.kv_scale, workspace=ws)
    assert mla.check_workspace(ws) == -9 and m.kept()
    mla.prefill_chunk(c.q, c.kv, c.table, c.lens, c.starts, SCALE, 0, m.out, m.lse, kv_scale=c.kv_scale, workspace=ws)
    assert mla.check_workspace(ws) == 0 and m.kept()
    chunk_cases.check(c, m.out, m.lse, what="after")


@pytest.mark.parametrize("starts", BAD)
@pytest.mark.parametrize("causal", [True, False])
def test_expanded_with_bad_starts(causal, starts):
    e = expanded_cases.make([40, 30, 20], [40, 30, 20], 4, causal, seed=32)
    q, kn, kr, v, qs, ks, _ = e.args
    ws, m = mla.make_prefill_workspace(q), Margins(90, 4, 128)
    for a, b in ((ints(starts), ks), (qs, ints(starts)), (ints(starts), ints(starts))):
        mla.prefill_expanded(q, kn, kr, v, a, b, causal, SCALE, 0, m.out, m.lse, workspace=ws)
        assert mla.check_workspace(ws) == -9 and m.kept()
    mla.prefill_expanded(q, kn, kr, v, qs, ks, causal, SCALE, 0, m.out, m.lse, workspace=ws)
    assert mla.check_workspace(ws) == 0 and m.kept()
    expanded_cases.check(e, m.out, m.lse, what="after")


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [2, 16])
def test_a_bad_page_or_length_spoils_its_own_request_only(kv_dtype, heads):
    """300 and 100 tokens around the bad request: one block of rows each (2 heads), or several."""
    lens, news = [300, 200, 100], [40, 30, 20]
    c = chunk_cases.make(lens, news, heads, kv_dtype, seed=30)
    good, rows, starts = c.table.clone(), rows_of(c), c.starts.tolist()
    ws, m = mla.make_prefill_workspace(c.q), Margins(90, heads, 512)

    def others():
        for b in (0, 2):
            s, n, t = starts[b], news[b], torch.arange(lens[b], device="cuda")
            kv = rows[good[b, t // 64].long(), t % 64]
            last = lens[b] - n + 1 + torch.arange(n, device="cuda")
            check_attention(c.q[s:s + n], kv, kv[:, :512], last, m.out[s:s + n], m.lse[s:s + n], 0, kv_dtype == "e4m3",
                            f"request {b}")

    def call():
        m.out.fill_(7)
        m.lse.fill_(7)
        mla.prefill_chunk(c.q, c.kv, c.table, c.lens, c.starts, SCALE, 0, m.out, m.lse, kv_scale=c.kv_scale, workspace=ws)
        return mla.check_workspace(ws)
    for column in (0, 2, 3):
        for bad in (-1, c.kv.shape[0], 2**31 - 1, -2**31):
            c.table[1, column] = bad
            assert call() == -9 and m.kept()
            others()
            c.table.copy_(good)
    for bad in (-5, c.table.shape[1] * 64 + 1, 2**31 - 1, -2**31):
        c.lens[1] = bad
        assert call() == -9 and m.kept()
        others()
    c.lens[1] = 200
    assert call() == 0
    chunk_cases.check(c, m.out, m.lse)
