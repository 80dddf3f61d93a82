"""prefill_expanded over tensors laid out otherwise than token by token: queries
inside wider rows, heads outermost, gaps, one token or head; offsets that pass 32
bits; the layouts it refuses."""
import pytest
import torch

import mla_paged_decode_gb300 as mla
from chunk_cases import SCALE, buffers, check_attention, ints
from expanded_cases import check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    mla.load_library()


def inside(t, width, at):
    """t's rows as part of rows of `width` values, the others NaN."""
    wide = torch.full((*t.shape[:-1], width), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., at:at + t.shape[-1]] = t
    return wide[..., at:at + t.shape[-1]]


def heads_first(t):
    """The same tensor with the heads outermost in memory."""
    return t.transpose(0, 1).contiguous().transpose(0, 1)


def spaced(t, step):
    """The same tensor with every row `step` tokens after the one before."""
    wide = torch.full((t.shape[0] * step, *t.shape[1:]), float("nan"), dtype=t.dtype, device=t.device)
    wide[::step] = t
    return wide[::step]


LAYOUTS = {
    "contiguous": lambda t: t.contiguous(),
    "wider rows": lambda t: inside(t, 328, 72),
    "heads first": heads_first,
    "heads first in wider rows": lambda t: heads_first(inside(t, 264, 8)) if t.dim() == 3 else inside(t, 264, 8),
    "every third token": lambda t: spaced(t, 3),
}


def again(c, layout, which, out, lse):
    """The call with the tensors in `which` in that layout; the others as they were."""
    t = list(c.args)
    for i in which:
        if t[i].dim() == 3 or "heads first" != layout:
            t[i] = LAYOUTS[layout](t[i])
            assert torch.equal(t[i], c.args[i])
    o2, l2 = buffers(c.q, 128)
    ws = mla.make_prefill_workspace(c.q)
    mla.prefill_expanded(*t, SCALE, 0, o2, l2, workspace=ws)
    assert mla.check_workspace(ws) == 0 and torch.equal(o2, out) and torch.equal(l2, lse), (layout, which)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [1, 5])
@pytest.mark.parametrize("news,keys", [([300, 1, 130], [300, 200, 131]), ([1], [1]), ([1], [300]), ([700], [1])])
def test_layouts(news, keys, heads, causal):
    """The same bits whatever the layout of each tensor."""
    c = make(news, keys, heads, causal, seed=40)
    out, lse = run(c)
    check(c, out, lse)
    for layout in LAYOUTS:
        for which in ((0,), (1,), (2,), (3,), (0, 1, 2, 3)):
            again(c, layout, which, out, lse)


def test_keys_and_values_past_four_gib():
    """Rows of keys, values and rope parts at offsets that pass 32 bits, bytes and values."""
    c = make([200, 70], [400, 333], 4, True, seed=41)
    M, step = c.up.shape[0], 4_400_000     # values from a token to the next: 733 * 4.4e6 = 3.2e9
    flat = torch.empty(M * step, dtype=torch.bfloat16, device="cuda")
    rows = flat.view(M, step)
    kn, v, kr = (rows[:, a:a + n] for a, n in ((0, 512), (1024, 512), (4096, 64)))
    kn, v = kn.unflatten(1, (4, 128)), v.unflatten(1, (4, 128))
    kn.copy_(c.up[..., :128])
    v.copy_(c.up[..., 128:])
    kr.copy_(c.latent[:, 512:])
    assert kn.stride() == (step, 128, 1) and (M - 1) * step > 2**31
    out, lse = run(c)
    check(c, out, lse)
    o2, l2 = buffers(c.q, 128)
    mla.prefill_expanded(c.q, kn, kr, v, c.q_starts, c.k_starts, True, SCALE, 0, o2, l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    del flat, rows, kn, v, kr
    # the heads outermost, a head's keys 4 GiB and more after those of the one before
    wide = torch.empty(4, 800_000_000, dtype=torch.bfloat16, device="cuda")
    kn = wide[:, :M * 128].unflatten(1, (M, 128)).transpose(0, 1)
    kn.copy_(c.up[..., :128])
    assert kn.stride() == (128, 800_000_000, 1) and 3 * kn.stride(1) > 2**31
    o2.fill_(7)
    mla.prefill_expanded(c.q, kn, c.latent[:, 512:], c.up[..., 128:], c.q_starts, c.k_starts, True, SCALE, 0, o2, l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("heads,tokens", [(128, 140_000), (1, 17_000_000)])
def test_queries_and_outputs_past_2_to_31_values(heads, tokens):
    """The last request's rows lie behind 2^31 values of out and more of q; the first
    request's queries, in front, see nothing of it."""
    c = make([300, 129], [260, 300], heads, False, seed=42)
    n0, n1 = 300, 129
    q = torch.zeros(tokens, heads, 192, dtype=torch.bfloat16, device="cuda")
    q[:n0], q[tokens - n1:] = c.q[:n0], c.q[n0:]
    out = torch.zeros(tokens, heads, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(tokens, heads, device="cuda")
    assert (tokens - n1) * heads * 128 > 2**31
    _, kn, kr, v, _, ks, _ = c.args
    starts, ks = ints([0, n0, tokens - n1, tokens]), ints([0, 260, 260, 560])
    ws = mla.make_prefill_workspace(q)
    # the request between has no keys: its rows are the neutral pair
    mla.prefill_expanded(q, kn, kr, v, starts, ks, False, SCALE, 0, out, lse, workspace=ws)
    assert mla.check_workspace(ws) == 0
    o2, l2 = buffers(c.q, 128)
    for a, b in ((slice(0, n0), slice(0, n0)), (slice(n0, None), slice(tokens - n1, tokens))):
        o2[a], l2[a] = out[b], lse[b]
    check(c, o2, l2)
    assert not out[n0:tokens - n1].any() and torch.isneginf(lse[n0:tokens - n1]).all()


def test_many_keyed_queries_far_back():
    """The same with keys for the rows between: every 1,000th is checked."""
    heads, tokens = 128, 140_000
    c = make([1], [129], heads, False, seed=43)
    q = torch.randn(tokens, heads, 192, device="cuda", dtype=torch.bfloat16)
    out, lse = torch.empty(tokens, heads, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(tokens, heads, device="cuda")
    _, kn, kr, v, *_ = c.args
    mla.prefill_expanded(q, kn, kr, v, ints([0, tokens]), ints([0, 129]), False, SCALE, 0, out, lse)
    some = torch.cat([torch.arange(0, tokens, 1000), torch.arange(tokens - 5, tokens)]).cuda()
    k = torch.cat([kn, kr[:, None].expand(-1, heads, 64)], -1)
    check_attention(q[some], k, v, torch.full_like(some, 129), out[some], lse[some], 0, what="some")


def test_layouts_that_are_refused():
    c = make([70], [130], 3, True, seed=44)
    q, kn, kr, v, *rest = c.args
    out, lse = buffers(c.q, 128)
    call = lambda *t: mla.prefill_expanded(*t, *rest, SCALE, 0, out, lse)  # noqa: E731
    one = kn[:, :1].expand(-1, 3, -1)                    # one key for all heads: a stride of 0
    for bad in ((q, one, kr, v), (q, kn, kr, one), (q, kn, kr[:1].expand(130, 64), v), (q[:1].expand(70, 3, 192), kn, kr, v),
                (inside(q, 196, 0), kn, kr, v), (q, inside(kn, 132, 4), kr, v), (q, kn, inside(kr, 132, 0), v),
                (inside(q, 200, 4), kn, kr, v)):         # strides and places that are no multiples of 8 values
        with pytest.raises(mla.MlaError):
            call(*bad)
    for bad in ((q.flip(0).transpose(1, 2).contiguous().transpose(1, 2), kn, kr, v),
                (q, kn, kr.t().contiguous().t(), v)):    # values of a row that are not consecutive
        with pytest.raises(ValueError, match="consecutive"):
            call(*bad)
    assert (out == 7).all() and (lse == 7).all()
