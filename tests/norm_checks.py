"""2-norms of attention outputs, request by request and head by head.

The element-wise limits of chunk_cases add up the largest errors that the
formats allow, so that over thousands of keys they are far wider than what a
right kernel does: a lost value row or coarse weights stay below them.  Here the
roundings are added up as what they are, independent of one another.

A rounding of relative step 2^-7 (bf16) is off by a number spread evenly over
one step: 2^-7 / sqrt(12) of the value in the root mean square at most, U.

* out: sum over the keys of (U p)^2 |v|^2 for the weights' rounding, and (U out)^2
  for the output's own.  An e4m3 cache's weights are an e4m3 and an e5m2 term:
  down to 2^-6 of the row's largest weight 2^-3 / sqrt(12) and 2^-2 / sqrt(12)
  multiplied, below it an even 2^-9 of the largest for the first term, and once the
  first term is zero (2^-10) the second's alone, 2^-2 / sqrt(12) of the weight;
  2^-16 / sqrt(12) of the largest where the second term ends.  1.25 times the root
  of the sum is allowed, for sums of finitely many roundings (a mean over evenly
  spread significands is 0.73 of it).
* lse: a score is a sum of dims / 16 products of 16 terms, each addition off by
  2^-23 of a partial sum, which is no larger than the request's largest score; twice
  that, and a few roundings of the result.  An e4m3 cache leaves out the part of q
  below its two terms, 2^-17 of the row's largest |q| a value: to first order the lse
  moves by its product with the mean key, sum p k.
"""
from __future__ import annotations

import math

import torch

from chunk_cases import SCALE, rows_of

U = 2.0**-7 / math.sqrt(12)


def weight_errors(p, top, e4m3):
    """Root mean square of the errors of weights p of which `top` is the row's largest."""
    if not e4m3:
        return U * p
    r12 = 1 / math.sqrt(12)
    normal = 2.0**-5 * r12 * r12 * p
    below = torch.minimum(2.0**-11 * r12 * r12 * top, 2.0**-2 * r12 * p)
    return torch.where(p >= 2.0**-6 * top, normal, below) + 2.0**-16 * r12 * top


def check_norms(q, k, v, last, out, lse, base=0, e4m3=False, what=""):
    """Rows q [n, H, D] over keys k [m, D] or [m, H, D] and values v alike, of which
    row i sees the first last[i] (one at least)."""
    n, H, D = q.shape
    lse = lse.double() * (math.log(2.0) if base else 1.0)
    worst = [0.0, 0.0]
    for h in range(H):
        kh, vh = (k if k.dim() == 2 else k[:, h]).double(), (v if v.dim() == 2 else v[:, h]).double()
        d2 = lim2 = dl2 = ll2 = 0.0
        for i0 in range(0, n, 256):
            rows = slice(i0, min(n, i0 + 256))
            qi, li = q[rows, h].double(), last[rows]
            hide = torch.arange(kh.shape[0], device=q.device) >= li[:, None]
            x = (qi @ kh.T * SCALE).masked_fill(hide, -math.inf)
            want_lse = torch.logsumexp(x, -1)
            p = torch.exp(x - want_lse[:, None])
            want = p @ vh
            e = weight_errors(p, p.amax(-1, keepdim=True), e4m3).masked_fill(hide, 0)
            d2 += float((out[rows, h].double() - want).square().sum())
            lim2 += float(e.square().sum(0) @ vh.square().sum(-1)) + float((U * want).square().sum())
            top = x.masked_fill(hide, 0).abs().amax()
            s = 2.0**-23 * (2 * (D // 16) * top + 4 * want_lse.abs()) + 2.0**-20
            if e4m3:
                s = s + 2.0**-17 * qi.abs().amax(-1) * (p @ kh).norm(dim=-1) * SCALE
            dl2 += float((lse[rows, h] - want_lse).square().sum())
            ll2 += float(s.square().sum())
        worst = [max(worst[0], math.sqrt(d2 / lim2) / 1.25), max(worst[1], math.sqrt(dl2 / ll2))]
        assert worst[0] <= 1, f"{what}: head {h}: out's error is {worst[0]:.2f} of what roundings give"
        assert worst[1] <= 1, f"{what}: head {h}: lse's error is {worst[1]:.2f} of what roundings give"
    return worst


def check_chunk(c, out, lse, base=0, what="", least=500):
    """A ChunkCase's requests of `least` tokens or more."""
    rows, starts, worst = rows_of(c), c.starts.tolist(), [0.0, 0.0]
    for b, L in enumerate(c.lens.tolist()):
        s, n = starts[b], starts[b + 1] - starts[b]
        if n == 0 or L - n + 1 < least:
            continue
        t = torch.arange(L, device=c.q.device)
        kv = rows[c.table[b, t // 64].long(), t % 64]
        last = L - n + 1 + torch.arange(n, device=c.q.device)
        w = check_norms(c.q[s:s + n], kv, kv[:, :512], last, out[s:s + n], lse[s:s + n], base,
                        c.kv.dtype == torch.uint8, f"{what} request {b}")
        worst = [max(a, b) for a, b in zip(worst, w)]
    assert worst[0] > 0, "no request is long enough"
    return worst


def check_expanded(c, out, lse, base=0, what="", least=500):
    qs, ks, worst = c.q_starts.tolist(), c.k_starts.tolist(), [0.0, 0.0]
    for b in range(len(qs) - 1):
        n, m = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
        if n == 0 or m - n + 1 < least:
            continue
        up, rope = c.up[ks[b]:ks[b + 1]], c.latent[ks[b]:ks[b + 1], None, 512:]
        k = torch.cat([up[..., :128], rope.expand(m, up.shape[1], 64)], -1)
        i = torch.arange(n, device=c.q.device)
        last = m - n + 1 + i if c.causal else torch.full_like(i, m)
        rows = slice(qs[b], qs[b + 1])
        w = check_norms(c.q[rows], k, up[..., 128:], last, out[rows], lse[rows], base, what=f"{what} request {b}")
        worst = [max(a, b) for a, b in zip(worst, w)]
    assert worst[0] > 0, "no request is long enough"
    return worst
