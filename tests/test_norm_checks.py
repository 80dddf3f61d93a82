"""The checks of 2-norms themselves, on the CPU: outputs with the formats'
roundings pass, outputs with a mistake over long contexts do not."""
import math

import pytest
import torch

from chunk_cases import SCALE
from norm_checks import check_norms

SIZES = [(20000, 576, 512, False), (20000, 576, 512, True), (5000, 192, 128, False), (700, 576, 512, True)]


def inputs(m, D, dv, e4m3, seed=0, n=40):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(m, D, generator=g)
    scale = 5.5 / 448
    k = (k / scale).to(torch.float8_e4m3fn).double() * scale if e4m3 else k.to(torch.bfloat16).double()
    v = k[:, :dv] if D == 576 else torch.randn(m, dv, generator=g).to(torch.bfloat16).double()
    q = torch.randn(n, 1, D, generator=g).to(torch.bfloat16)
    return q, k, v, m - n + 1 + torch.arange(n)


def two_terms(e):
    hi = e.float().to(torch.float8_e4m3fn).float()
    return (hi + (e.float() - hi).to(torch.float8_e5m2).float()).double()


def attend(q, k, v, last, e4m3, shift=0.0, weights=None, mask=0, coarse=False):
    """out, lse as a kernel rounds them; `shift`: how far its maximum lies below the row's
    (base 2); `weights`: a change to the weights; `mask`: keys seen too many."""
    x = q[:, 0].double() @ k.T * SCALE
    x = x.masked_fill(torch.arange(k.shape[0]) >= (last + mask)[:, None], -math.inf)
    top = x.amax(-1, keepdim=True) - shift * math.log(2)
    e = torch.exp(x - top)
    if weights is not None:
        e = weights(e, last)
    r = two_terms(e) if e4m3 else e.to(torch.bfloat16).double()
    if coarse:  # 4 significant bits
        f, s = torch.frexp(e)
        r = torch.ldexp((f * 16).round() / 16, s)
    out = (r @ v) / (r if e4m3 else e).sum(-1, keepdim=True)
    lse = torch.log(e.sum(-1)) + top[:, 0]
    return out.to(torch.bfloat16)[:, None], lse.float()[:, None]


@pytest.mark.parametrize("m,D,dv,e4m3", SIZES)
@pytest.mark.parametrize("shift", [0.0, 3.3, 8.0])
def test_roundings_pass(m, D, dv, e4m3, shift):
    for seed in range(3):
        a = inputs(m, D, dv, e4m3, seed)
        out, lse = attend(*a, e4m3, shift)
        worst = check_norms(*a, out, lse, e4m3=e4m3)
        assert worst[0] > 0.3   # and by less than a factor of three
    a = inputs(m, D, dv, e4m3, 9, n=1)
    check_norms(*a, *attend(*a, e4m3, shift), e4m3=e4m3)


def lose(rows):
    def f(e, last):
        e = e.clone()
        e[:, rows] = 0
        return e
    return f


def lose_own(e, last):
    e = e.clone()
    e[torch.arange(len(last)), last - 1] = 0
    return e


MISTAKES = {"one token too many": dict(mask=1), "one token too few": dict(mask=-1), "its own token": dict(weights=lose_own),
            "a lost key": dict(weights=lose([77])), "eight lost keys": dict(weights=lose(list(range(64, 72)))),
            "coarse weights": dict(coarse=True)}


@pytest.mark.parametrize("m,D,dv,e4m3", SIZES)
@pytest.mark.parametrize("name", MISTAKES)
def test_mistakes_do_not(m, D, dv, e4m3, name):
    q, k, v, last = inputs(m + 1, D, dv, e4m3, 1)
    last = last - 1          # so that a key too many exists
    out, lse = attend(q, k, v, last, e4m3, **MISTAKES[name])
    with pytest.raises(AssertionError, match="of what roundings give"):
        check_norms(q, k, v, last, out, lse, e4m3=e4m3)


@pytest.mark.parametrize("m,D,dv,e4m3", SIZES)
@pytest.mark.parametrize("rows", [[300], list(range(64, 72))])
def test_lost_value_rows_do_not(m, D, dv, e4m3, rows):
    """Value rows of zeros: the lse does not show them."""
    q, k, v, last = inputs(m, D, dv, e4m3, 2)
    w = v.clone()
    w[rows] = 0
    out, lse = attend(q, k, w, last, e4m3)
    with pytest.raises(AssertionError, match="out's error"):
        check_norms(q, k, v, last, out, lse, e4m3=e4m3)
