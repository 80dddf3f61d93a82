"""Cases and the 64-bit reference of decode_window and decode_shared.

Rows that no query of a request sees (page tails, tokens out of a window,
pages nobody owns) hold NaN, and table entries of pages out of view are -1: a
correct kernel lets none of them into its outputs.

Tolerances, from the formats' roundings alone (half a step: bf16 2^-8):

* scores: fp32 sums of 576 products, each addition off by 2^-23 of the sum of
  magnitudes at most (the tensor core may truncate); an e4m3 cache adds the
  part of q below its two e4m3 terms, 2^-17 of the group's largest |q|;
* weights: bf16, 2^-8 each; e4m3: 2^-7 down to 2^-6 of the maximum, 2^-3
  below it, and 2^-17 of the maximum for the smallest;
* out = sum w v / sum w: twice the weights' error times sum p |v|, plus the
  output's own rounding; lse: the scores' error plus fp32 roundings.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

import mla_paged_decode_gb300 as mla
import workloads

SCALE = workloads.SM_SCALE_192


@dataclass
class ViewCase:
    q: torch.Tensor
    kv: torch.Tensor
    kv_scale: float
    table: torch.Tensor
    lens: torch.Tensor
    seen: list  # per request and query token: indices of the tokens it sees


def _rows(c):
    x = c.kv.view(torch.float8_e4m3fn).double() * c.kv_scale if c.kv.dtype == torch.uint8 else c.kv.double()
    return x


def make(lens, heads, q_len, kv_dtype, seen_of, seed, device="cuda", shared=None, spare=3, q_gain=1.0,
         width=0):
    """seen_of(L, i): token indices query token i of a request of length L
    sees.  shared: (group_starts, shared_pages) as lists.  width: columns of
    the block table, at least."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-L // 64) for L in lens]
    sp = [0] * len(lens)
    if shared:
        starts, pages = shared
        for k, n in enumerate(pages):
            for b in range(starts[k], starts[k + 1]):
                sp[b] = n
    width = max(1, width, max(need, default=1), max(sp, default=1))
    total = sum(max(0, n - s) for n, s in zip(need, sp)) + (sum(shared[1]) if shared else 0) + spare
    perm = torch.randperm(total, generator=g).to(torch.int32)
    kv = torch.randn(total, 64, 576, generator=g)
    scale = 1.0
    if kv_dtype == "e4m3":
        scale = float(kv.abs().max()) / 448.0
        kv = (kv / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        kv = kv.to(torch.bfloat16)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    if shared:
        for k, n in enumerate(pages):
            table[starts[k]:starts[k + 1], :n] = perm[at:at + n]
            at += n
    for b, n in enumerate(need):
        if n > sp[b]:
            table[b, sp[b]:n] = perm[at:at + n - sp[b]]
            at += n - sp[b]
    seen = [[seen_of(L, i) for i in range(q_len)] for L in lens]
    keep = torch.zeros(total, 64, dtype=torch.bool)
    if shared:  # the shared pages hold a finished prompt
        for k, n in enumerate(pages):
            if starts[k] < starts[k + 1]:
                keep[table[starts[k], :n].long()] = True
    for b in range(len(lens)):
        t = torch.unique(torch.cat(seen[b]))
        keep[table[b, t // 64].long(), t % 64] = True
        out = torch.ones(width, dtype=torch.bool)
        out[t // 64] = False
        out[:sp[b]] = False
        table[b, out] = -1
    if kv_dtype == "e4m3":
        kv[~keep] = 0x7F
    else:
        kv[~keep] = math.nan
    q = (torch.randn(len(lens), q_len, heads, 576, generator=g) * q_gain).to(torch.bfloat16)
    return ViewCase(q.to(device), kv.to(device), scale, table.to(device),
                    torch.tensor(lens, dtype=torch.int32, device=device), seen)


def window_seen(window, sinks, q_len):
    def f(L, i):
        pos = L - q_len + i
        t = torch.arange(max(0, pos + 1))
        return t[(t > pos - window) | (t < sinks)]
    return f


def causal_seen(q_len):
    return lambda L, i: torch.arange(max(0, L - q_len + i + 1))


def check(c: ViewCase, out, lse, base=0, what=""):
    """out / lse against the definition in 64 bits, element by element."""
    rows = _rows(c)
    e4m3 = c.kv.dtype == torch.uint8
    B, T, H, _ = c.q.shape
    assert not torch.isnan(out).any() and not torch.isnan(lse).any(), f"{what}: NaN"
    lse = lse.double() * (math.log(2.0) if base else 1.0)
    qmax = c.q.double().abs().max()
    for b in range(B):
        for i in range(T):
            t = c.seen[b][i].to(c.kv.device)
            if t.numel() == 0:
                assert (out[b, i] == 0).all() and torch.isneginf(lse[b, i]).all(), f"{what}: request {b}"
                continue
            kv = rows[c.table[b, t // 64].long(), t % 64]
            q = c.q[b, i].double()
            x = q @ kv.T * SCALE
            eps = 576 * 2.0**-23 * (q.abs() @ kv.abs().T).amax(-1) * SCALE
            if e4m3:
                eps = eps + 2.0**-17 * qmax * kv.abs().sum(-1).max() * SCALE
            want_lse = torch.logsumexp(x, -1)
            d = (lse[b, i] - want_lse).abs()
            # log2 and its scaling round the LSE's own size; exp2 is good to 2^-20
            lim = eps + 2.0**-20 + 2.0**-21 * (want_lse.abs() + x.abs().amax(-1))
            assert (d <= lim).all(), f"{what}: request {b} token {i}: lse off by {d.max():.3e} (limit {lim.min():.3e})"
            p = torch.softmax(x, -1)
            want = p @ kv[:, :512]
            w = 2.0**-8 * p
            if e4m3:
                top = p.amax(-1, keepdim=True)
                w = torch.where(p >= 2.0**-6 * top, 2.0**-7, 2.0**-3) * p + 2.0**-17 * top
            # the normaliser carries the weights' error too
            err = w @ kv[:, :512].abs() + w.sum(-1, keepdim=True) * want.abs()
            err = err + 2 * (eps[:, None] + 2.0**-18) * (p @ kv[:, :512].abs())
            lim = 2.0**-8 * (want.abs() + err) + err
            d = (out[b, i].double() - want).abs()
            assert (d <= lim).all(), (f"{what}: request {b} token {i}: out off by {d.max():.3e}, "
                                      f"{(d / lim).max():.2f} of the limit")


def buffers(c):
    B, T, H, _ = c.q.shape
    out = torch.full((B, T, H, 512), math.nan, dtype=torch.bfloat16, device=c.q.device)
    return out, torch.full((B, T, H), math.nan, dtype=torch.float32, device=c.q.device)


def run_window(c, window, sinks, base=0, ws=None, stream=None):
    out, lse = buffers(c)
    ws = ws if ws is not None else mla.make_workspace(c.q, c.kv, c.table, c.kv_scale)
    mla.decode_window(c.q, c.kv, c.table, c.lens, window, sinks, SCALE, base, out, lse,
                      kv_scale=c.kv_scale, workspace=ws, stream=stream)
    assert mla.check_workspace(ws, stream) == 0
    return out, lse


def run_shared(c, starts, pages, base=0, ws=None, stream=None):
    out, lse = buffers(c)
    dev = c.q.device
    ws = ws if ws is not None else mla.make_shared_workspace(c.q, c.kv, c.table, len(pages), c.kv_scale)
    mla.decode_shared(c.q, c.kv, c.table, c.lens, torch.tensor(starts, dtype=torch.int32, device=dev),
                      torch.tensor(pages, dtype=torch.int32, device=dev), SCALE, base, out, lse,
                      kv_scale=c.kv_scale, workspace=ws, stream=stream)
    assert mla.check_workspace(ws, stream) == 0
    return out, lse
