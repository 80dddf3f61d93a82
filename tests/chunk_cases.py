"""Cases and the 64-bit definitions of the chunk operators.

A ragged batch: request b has lens[b] cached tokens, the last news[b] of them
new; `pad` rows at the end belong to nobody and keep what they hold.  Cache
rows past a request's length, pages nobody owns and table entries past a
request's pages hold NaN or -1: a correct kernel lets none of them through.

Tolerances, from the formats' roundings alone (half a step: bf16 2^-8), as in
view_cases: scores are fp32 sums of 576 (expanded: 192) products, each
addition off by 2^-23 of the sum of magnitudes at most, an e4m3 cache adding
the part of q below its two e4m3 terms, 2^-17 of the row's largest |q|; weights
are bf16, 2^-8 each (e4m3: 2^-7 down to 2^-6 of the maximum, 2^-3 below it,
2^-17 of the maximum for the smallest); out = sum w v / sum w carries twice the
weights' error times sum p |v| and its own rounding.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

import mla_paged_decode_gb300 as mla
import workloads

SCALE = workloads.SM_SCALE_192


@dataclass
class ChunkCase:
    q: torch.Tensor
    kv: torch.Tensor
    kv_scale: float
    table: torch.Tensor
    lens: torch.Tensor
    starts: torch.Tensor


def ints(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def starts_of(news, first=0):
    s = [first]
    for n in news:
        s.append(s[-1] + n)
    return s


def make(lens, news, heads, kv_dtype, seed, pad=0, device="cuda", spare=3, q_gain=1.0, width=0):
    g = torch.Generator().manual_seed(seed)
    need = [-(-L // 64) for L in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g).to(torch.int32)
    kv = torch.randn(total, 64, 576, generator=g)
    scale = 1.0
    if kv_dtype == "e4m3":
        scale = float(kv.abs().max()) / 448.0
        kv = (kv / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        kv = kv.to(torch.bfloat16)
    table = torch.full((len(lens), max(1, width, max(need, default=1))), -1, dtype=torch.int32)
    keep = torch.zeros(total, 64, dtype=torch.bool)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
        t = torch.arange(lens[b])
        keep[table[b, t // 64].long(), t % 64] = True
    kv[~keep] = 0x7F if kv_dtype == "e4m3" else math.nan
    q = (torch.randn(sum(news) + pad, heads, 576, generator=g) * q_gain).to(torch.bfloat16)
    return ChunkCase(q.to(device), kv.to(device), scale, table.to(device), ints(lens, device),
                     ints(starts_of(news), device))


def buffers(q, dim=512):
    n, heads, _ = q.shape
    out = torch.full((n, heads, dim), 7.0, dtype=torch.bfloat16, device=q.device)
    return out, torch.full((n, heads), 7.0, dtype=torch.float32, device=q.device)


def run(c, base=0, ws=None, stream=None):
    out, lse = buffers(c.q)
    ws = ws if ws is not None else mla.make_prefill_workspace(c.q)
    mla.prefill_chunk(c.q, c.kv, c.table, c.lens, c.starts, SCALE, base, out, lse, kv_scale=c.kv_scale, workspace=ws,
                      stream=stream)
    assert mla.check_workspace(ws, stream) == 0
    return out, lse


def check_attention(q, k, v, last, out, lse, base, e4m3=False, what=""):
    """Rows q [n, H, D] over keys k [m, D] or [m, H, D] and values v alike, of
    which row i sees the first last[i], element by element in 64 bits."""
    n, H, D = q.shape
    assert not torch.isnan(out).any() and not torch.isnan(lse).any(), f"{what}: NaN"
    lse = lse.double() * (math.log(2.0) if base else 1.0)
    for h in range(H):
        kh = (k if k.dim() == 2 else k[:, h]).double()
        vh = (v if v.dim() == 2 else v[:, h]).double()
        for i0 in range(0, n, 512):
            qi, li = q[i0:i0 + 512, h].double(), last[i0:i0 + 512]
            o, w_lse = out[i0:i0 + 512, h].double(), lse[i0:i0 + 512, h]
            none = li <= 0
            assert (o[none] == 0).all() and torch.isneginf(w_lse[none]).all(), f"{what}: head {h}: empty rows"
            if none.all():
                continue
            qi, li, o, w_lse = qi[~none], li[~none], o[~none], w_lse[~none]
            m = int(li.max())
            kk, vv = kh[:m], vh[:m]
            hide = torch.arange(m, device=q.device) >= li[:, None]
            x = (qi @ kk.T * SCALE).masked_fill(hide, -math.inf)
            eps = D * 2.0**-23 * (qi.abs() @ kk.abs().T).masked_fill(hide, 0).amax(-1) * SCALE
            if e4m3:
                eps = eps + 2.0**-17 * qi.abs().amax(-1) * kk.abs().sum(-1).max() * SCALE
            want_lse = torch.logsumexp(x, -1)
            lim = eps + 2.0**-20 + 2.0**-21 * (want_lse.abs() + x.masked_fill(hide, 0).abs().amax(-1))
            d = (w_lse - want_lse).abs()
            assert (d <= lim).all(), f"{what}: head {h}: lse off by {d.max():.3e} (limit {lim.min():.3e})"
            p = torch.softmax(x, -1)
            want = p @ vv
            w = 2.0**-8 * p
            if e4m3:
                top = p.amax(-1, keepdim=True)
                w = torch.where(p >= 2.0**-6 * top, 2.0**-7, 2.0**-3) * p + 2.0**-17 * top
                w = w.masked_fill(hide, 0)
            err = w @ vv.abs() + w.sum(-1, keepdim=True) * want.abs()
            err = err + 2 * (eps[:, None] + 2.0**-18) * (p @ vv.abs())
            lim = 2.0**-8 * (want.abs() + err) + err
            d = (o - want).abs()
            assert (d <= lim).all(), f"{what}: head {h}: out off by {d.max():.3e}, {(d / lim).max():.2f} of the limit"


def rows_of(c):
    return c.kv.view(torch.float8_e4m3fn).double() * c.kv_scale if c.kv.dtype == torch.uint8 else c.kv.double()


def check(c, out, lse, base=0, what=""):
    rows, starts = rows_of(c), c.starts.tolist()
    for b, L in enumerate(c.lens.tolist()):
        s, n = starts[b], starts[b + 1] - starts[b]
        if n == 0:
            continue
        t = torch.arange(L, device=c.q.device)
        kv = rows[c.table[b, t // 64].long(), t % 64]
        last = L - n + 1 + torch.arange(n, device=c.q.device)
        check_attention(c.q[s:s + n], kv, kv[:, :512], last, out[s:s + n], lse[s:s + n], base,
                        c.kv.dtype == torch.uint8, f"{what} request {b}")
    for part in (slice(0, starts[0]), slice(starts[-1], None)):
        assert (out[part] == 7).all() and (lse[part] == 7).all(), f"{what}: rows of nobody"
