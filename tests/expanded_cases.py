"""Cases of prefill_expanded, checked with chunk_cases.check_attention.  The
keys are parts of wider rows, as a program has them; rows of nobody hold NaN."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

import mla_paged_decode_gb300 as mla
from chunk_cases import SCALE, buffers, check_attention, ints, starts_of


@dataclass
class ExpandedCase:
    q: torch.Tensor
    up: torch.Tensor       # [M, H, 256]: keys, then values
    latent: torch.Tensor   # [M, 576]: the last 64 the rope part
    q_starts: torch.Tensor
    k_starts: torch.Tensor
    causal: bool

    @property
    def args(self):
        return (self.q, self.up[..., :128], self.latent[:, 512:], self.up[..., 128:], self.q_starts, self.k_starts,
                self.causal)


def make(news, keys, heads, causal, seed, pad=0, q_gain=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    M = sum(keys) + pad
    q = (torch.randn(sum(news) + pad, heads, 192, generator=g) * q_gain).to(torch.bfloat16)
    up = torch.randn(M, heads, 256, generator=g).to(torch.bfloat16)
    latent = torch.randn(M, 576, generator=g).to(torch.bfloat16)
    up[sum(keys):], latent[sum(keys):] = math.nan, math.nan
    return ExpandedCase(q.to(device), up.to(device), latent.to(device), ints(starts_of(news), device),
                        ints(starts_of(keys), device), causal)


def run(c, base=0, ws=None, stream=None):
    out, lse = buffers(c.q, 128)
    ws = ws if ws is not None else mla.make_prefill_workspace(c.q)
    mla.prefill_expanded(*c.args, SCALE, base, out, lse, workspace=ws, stream=stream)
    assert mla.check_workspace(ws, stream) == 0
    return out, lse


def check(c, out, lse, base=0, what="", skip=()):
    qs, ks = c.q_starts.tolist(), c.k_starts.tolist()
    for b in range(len(qs) - 1):
        n, m = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
        if n == 0 or b in skip:
            continue
        up, rope = c.up[ks[b]:ks[b + 1]], c.latent[ks[b]:ks[b + 1], None, 512:]
        k = torch.cat([up[..., :128], rope.expand(m, up.shape[1], 64)], -1)
        i = torch.arange(n, device=c.q.device)
        last = (m - n + 1 + i).clamp(min=0) if c.causal else torch.full_like(i, m)
        rows = slice(qs[b], qs[b + 1])
        check_attention(c.q[rows], k, up[..., 128:], last, out[rows], lse[rows], base, what=f"{what} request {b}")
    for part in (slice(0, qs[0]), slice(qs[-1], None)):
        assert (out[part] == 7).all() and (lse[part] == 7).all(), f"{what}: rows of nobody"
