"""Cases of the prefill side of the paged latent cache: a chunk of new tokens
written into the cache and read back, its attention over the cache (absorbed
form) and its attention over expanded keys and values.

Each case runs one pass of one operator: with ``own`` true through the
library's calls, otherwise in plain torch operations in fp32.  ``exact`` is
the definition in 64 bits.

Batches are ragged: request b's tokens are rows starts[b] .. starts[b + 1] of
the tensors that hold a row a token, and rows from starts[-1] on belong to
nobody (a batch padded to the size of a captured graph); they stay as they are.
"""
import math

import torch

own = False

PAGE, DQK, DV = 64, 576, 512          # the latent cache: 512 latent + 64 rope
NOPE, ROPE, DVX = 128, 64, 128        # an expanded head: 128 + 64 for the scores, 128 for the value
SM_SCALE = 1.0 / math.sqrt(192.0)
KV_SCALE = 5.5 / 448.0
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the prompt of one short request goes into the cache: latency
        dict(name="append_small", op="append", kv="bf16", batch=1, new_lo=48, new_hi=48, ctx_hi=0, ones=0, pad=0),
        # a step of a serving loop: 40 requests decode, 24 prefill, padded for a graph; e4m3 cache
        dict(name="append_mixed_e4m3", op="append", kv="e4m3", batch=64, new_lo=100, new_hi=1999, ctx_hi=8000,
             ones=40, pad=77),
        # eight long prompts at once
        dict(name="append_large", op="append", kv="bf16", batch=8, new_lo=8192, new_hi=8192, ctx_hi=700, ones=0,
             pad=0),
        # the context of one short conversation, to be expanded: latency
        dict(name="read_small", op="read", kv="bf16", batch=1, new_lo=300, new_hi=300, ctx_hi=0, ones=0, pad=0),
        # the contexts of 32 requests, each from where the last piece of its context ended; e4m3 cache
        dict(name="read_ragged_e4m3", op="read", kv="e4m3", batch=32, new_lo=1, new_hi=4095, ctx_hi=2000, ones=0,
             pad=33),
        # a short prompt of the small configuration (16 heads, 300 tokens in all): latency
        dict(name="chunk_small", op="chunk", kv="bf16", heads=16, batch=1, new_lo=48, new_hi=48, ctx_lo=252,
             ctx_hi=252, ones=0, pad=0),
        # a serving step with 16 heads on this GPU: 24 requests decode beside two chunks of prompts, padded
        dict(name="chunk_mixed", op="chunk", kv="bf16", heads=16, batch=26, new_lo=300, new_hi=1000, ctx_lo=500,
             ctx_hi=6000, ones=24, pad=19),
        # chunks of six requests, all 128 heads, e4m3 cache
        dict(name="chunk_ragged_e4m3", op="chunk", kv="e4m3", heads=128, batch=6, new_lo=1, new_hi=257, ctx_lo=1000,
             ctx_hi=8000, ones=0, pad=0),
        # two chunks of 1,024 tokens after 15K tokens of context, 64 heads
        dict(name="chunk_large", op="chunk", kv="bf16", heads=64, batch=2, new_lo=1024, new_hi=1024, ctx_lo=15360,
             ctx_hi=15360, ones=0, pad=0),
        # a first prompt of 200 tokens, 16 heads: latency
        dict(name="expanded_small", op="expanded", causal=True, heads=16, batch=1, new_lo=200, new_hi=200, ctx_lo=0,
             ctx_hi=0, ones=0, pad=0),
        # chunks against pieces of their earlier context (all of it seen), to be merged with their own part
        dict(name="expanded_context", op="expanded", causal=False, heads=64, batch=5, new_lo=100, new_hi=700,
             ctx_lo=0, ctx_hi=5000, ones=0, pad=13),
        # a prompt's last 2,048 tokens of 10,240, all 128 heads
        dict(name="expanded_large", op="expanded", causal=True, heads=128, batch=1, new_lo=2048, new_hi=2048,
             ctx_lo=8192, ctx_hi=8192, ones=0, pad=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "chunk", "chunk", "expanded", "expanded"])
    kv = rng.choice(["bf16", "e4m3"])
    pad = rng.choice([0, rng.randint(1, 200)])
    if op in ("append", "read"):
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 8192 * 8 // batch)
        ones = rng.choice([0, rng.randint(0, batch)])
        return dict(op=op, kv=kv, batch=batch, new_lo=rng.randint(1, hi), new_hi=hi, ctx_hi=rng.randint(0, 8000),
                    ones=ones, pad=pad)
    while True:
        hi, chi = _log_int(rng, 1, 2048), _log_int(rng, 1, 15360)
        batch = _log_int(rng, 1, 26)
        c = dict(op=op, heads=rng.choice([16, 64, 128, rng.randint(1, 128)]), batch=batch, new_lo=rng.randint(1, hi),
                 new_hi=hi, ctx_lo=rng.randint(0, chi), ctx_hi=chi, ones=rng.choice([0, 0, rng.randint(0, batch)]),
                 pad=pad)
        c.update(dict(kv=kv) if op == "chunk" else dict(causal=rng.random() < 0.6))
        # no more work or temporaries than the largest listed ones
        scores = batch * hi * c["heads"] * (chi + hi)
        if scores <= (2 * 1024 * 64 * 16384 if op == "chunk" else 128 * 2048 * 10240) and batch * (chi + hi) <= 130000:
            return c


# ---------------------------------------------------------------- inputs

class State:
    """What a serving loop holds: the cache, its tables and the call's buffers."""


def _generators(seed):
    c, g = torch.Generator(), torch.Generator(device=DEV)
    c.manual_seed(seed * 7919 + 17)
    g.manual_seed(seed * 104729 + 19)
    return c, g


def _lengths(case, gen=None):
    """New tokens of each request and the tokens before them: the same
    lengths for all inputs of a case, in another order for each."""
    g = torch.Generator()
    g.manual_seed(5)
    B = case["batch"]
    new = torch.randint(case["new_lo"], case["new_hi"] + 1, (B,), generator=g)
    new[:case["ones"]] = 1
    ctx = torch.randint(case.get("ctx_lo", 0), case["ctx_hi"] + 1, (B,), generator=g)
    order = torch.randperm(B, generator=gen) if gen else torch.arange(B)
    return new[order].tolist(), ctx[order].tolist()


def _starts(lens):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV)


def _normal(gen, *shape):
    return torch.empty(*shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)


def _cache(lens, kv, cpu, gen):
    """A pool of N(0, 1) rows, its pages dealt to requests of these lengths."""
    need = [-(-n // PAGE) for n in lens]
    perm = torch.randperm(sum(need) + 3, generator=cpu).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    x = _normal(gen, sum(need) + 3, PAGE, DQK)
    if kv == "e4m3":
        x = (x.float() / KV_SCALE).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x, table.to(DEV)


def prepare(case, seed):
    cpu, gen = _generators(seed)
    s = State()
    s.case = case
    new, ctx = _lengths(case, cpu)
    rows = sum(new) + case["pad"]
    s.new, s.ctx = new, ctx
    s.starts = _starts(new)
    s.scale = KV_SCALE if case.get("kv") == "e4m3" else 1.0
    s.divisor = torch.tensor(s.scale, device=DEV)  # (a division by a number becomes a product with its inverse)
    if case["op"] != "expanded":
        s.kv, s.table = _cache([n + c for n, c in zip(new, ctx)], case["kv"], cpu, gen)
        s.positions = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    if case["op"] == "append":
        s.rows = _normal(gen, rows, DQK)
    elif case["op"] == "read":
        s.out = torch.zeros(rows, DQK, dtype=torch.bfloat16, device=DEV)
    else:
        H = case["heads"]
        s.out = torch.zeros(rows, H, DV if case["op"] == "chunk" else DVX, dtype=torch.bfloat16, device=DEV)
        s.lse = torch.zeros(rows, H, dtype=torch.float32, device=DEV)
        if case["op"] == "chunk":
            s.lens = torch.tensor([n + c for n, c in zip(new, ctx)], dtype=torch.int32, device=DEV)
            s.q = _normal(gen, rows, H, DQK)
        else:
            s.keys = [n + c if case["causal"] else c for n, c in zip(new, ctx)]
            s.k_starts = _starts(s.keys)
            s.q = _normal(gen, rows, H, NOPE + ROPE)
            # one projection gives a token's keys and values of all heads; its
            # rope part lies in the latent row that it came from
            s.up = _normal(gen, sum(s.keys), H, NOPE + DVX)
            s.latent = _normal(gen, sum(s.keys), DQK)
    if own:
        import mla_paged_decode_gb300 as mla
        s.mla = mla
        if case["op"] in ("chunk", "expanded"):
            s.workspace = mla.make_prefill_workspace(s.q)
    return s


# ---------------------------------------------------------------- plain forms

def _tokens(starts, rows):
    """For each of the rows that belong to a request: its request and its
    number within the request."""
    i = torch.arange(rows, device=DEV)
    b = torch.searchsorted(starts[1:].contiguous(), i.to(torch.int32), right=True)
    return b, i - starts.long()[b]


def _slots(s, rows):
    """Cache row of each new token."""
    b, i = _tokens(s.starts, rows)
    t = s.positions.long()[b] + i
    return s.table[b, t // PAGE].long() * PAGE + t % PAGE


def _plain_append(s):
    rows = sum(s.new)
    x = s.rows[:rows]
    if s.case["kv"] == "e4m3":
        x = (x.float() / s.divisor).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s.kv.view(-1, DQK)[_slots(s, rows)] = x


def _plain_read(s):
    rows = sum(s.new)
    x = s.kv.view(-1, DQK)[_slots(s, rows)]
    if s.case["kv"] == "e4m3":
        x = (x.view(torch.float8_e4m3fn).float() * s.divisor).to(torch.bfloat16)
    s.out[:rows] = x


def _softmax(x, seen):
    """Weights (in place) and lse of scores x, of which `seen` count."""
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total == 0, torch.ones_like(total), total)
    return p, (top + torch.log(total)).squeeze(-1)


def _padded(s):
    """Row of each (request, new token), request by request; those past a
    request's tokens repeat a row and are not taken."""
    n = max(s.new)
    i = torch.arange(n, device=DEV)
    valid = i < (s.starts[1:] - s.starts[:-1])[:, None]
    return (s.starts[:-1, None] + i).clamp(max=s.q.shape[0] - 1).long(), valid


def _plain_chunk(s):
    B, H, n = s.case["batch"], s.case["heads"], max(s.new)
    rows, valid = _padded(s)
    width = s.table.shape[1]
    kv = s.kv[s.table.clamp(min=0).long()].view(B, width * PAGE, DQK)
    kv = kv.view(torch.float8_e4m3fn).float() * s.divisor if s.case["kv"] == "e4m3" else kv.float()
    q = s.q[rows].float().view(B, n * H, DQK)
    x = torch.bmm(q, kv.transpose(1, 2)).mul_(SM_SCALE).view(B, n, H, -1)
    last = s.positions[:, None] + torch.arange(n, device=DEV)
    seen = torch.arange(width * PAGE, device=DEV) <= last[..., None]
    p, lse = _softmax(x, seen[:, :, None, :])
    out = torch.bmm(p.view(B, n * H, -1), kv[..., :DV]).view(B, n, H, DV)
    s.out[rows[valid]] = out[valid].to(torch.bfloat16)
    s.lse[rows[valid]] = lse[valid]


def _plain_expanded(s):
    H, n, m = s.case["heads"], max(s.new), max(1, max(s.keys))
    rows, valid = _padded(s)
    j = torch.arange(m, device=DEV)
    lens = s.k_starts[1:] - s.k_starts[:-1]
    keys = (s.k_starts[:-1, None] + j).clamp(max=max(0, s.up.shape[0] - 1)).long()
    B = len(s.new)
    if s.up.shape[0] == 0:
        s.out[rows[valid]] = 0
        s.lse[rows[valid]] = -math.inf
        return
    up = s.up[keys].float().permute(0, 2, 1, 3)
    q = s.q[rows].float().permute(0, 2, 1, 3)
    x = torch.matmul(q[..., :NOPE], up[..., :NOPE].transpose(2, 3))
    x += torch.matmul(q[..., NOPE:], s.latent[keys][..., DV:].float().transpose(1, 2)[:, None])
    x *= SM_SCALE
    seen = (j < lens[:, None])[:, None, :].expand(B, n, m)
    if s.case["causal"]:
        seen = seen & (j <= (lens - (s.starts[1:] - s.starts[:-1]))[:, None, None]
                       + torch.arange(n, device=DEV)[:, None])
    p, lse = _softmax(x, seen[:, None])
    out = torch.matmul(p, up[..., NOPE:]).transpose(1, 2)
    s.out[rows[valid]] = out[valid].to(torch.bfloat16)
    s.lse[rows[valid]] = lse.transpose(1, 2)[valid]


# ---------------------------------------------------------------- one pass

def run(s):
    op = s.case["op"]
    if op == "append":
        if own:
            s.mla.kv_append_chunk(s.rows, s.kv, s.table, s.starts, s.positions, kv_scale=s.scale)
        else:
            _plain_append(s)
        return {"kv": s.kv if s.case["kv"] == "bf16" else s.kv.view(torch.float8_e4m3fn)}
    if op == "read":
        if own:
            s.mla.kv_read(s.kv, s.table, s.starts, s.positions, s.out, kv_scale=s.scale)
        else:
            _plain_read(s)
        return {"rows": s.out}
    if op == "chunk":
        if own:
            s.mla.prefill_chunk(s.q, s.kv, s.table, s.lens, s.starts, SM_SCALE, s.mla.LSE_NATURAL, s.out, s.lse,
                                kv_scale=s.scale, workspace=s.workspace)
        else:
            _plain_chunk(s)
    else:
        if own:
            s.mla.prefill_expanded(s.q, s.up[..., :NOPE], s.latent[:, DV:], s.up[..., NOPE:], s.starts, s.k_starts,
                                   s.case["causal"], SM_SCALE, s.mla.LSE_NATURAL, s.out, s.lse,
                                   workspace=s.workspace)
        else:
            _plain_expanded(s)
    return {"out": s.out, "lse": s.lse}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    new, ctx = _lengths(case)
    n = sum(new)
    row = DQK * (1 if case.get("kv") == "e4m3" else 2)
    if case["op"] in ("append", "read"):
        return {"bytes": n * (2 * DQK + row) + 4 * sum(-(-x // PAGE) for x in new), "flops": 0}
    H = case["heads"]
    if case["op"] == "chunk":
        seen = sum(x * c + x * (x + 1) // 2 for x, c in zip(new, ctx))
        return {"bytes": row * sum(x + c for x, c in zip(new, ctx)) + n * H * (2 * DQK + 2 * DV + 4),
                "flops": 2.0 * H * (DQK + DV) * seen}
    if case["causal"]:
        seen = sum(x * c + x * (x + 1) // 2 for x, c in zip(new, ctx))
        keys = sum(new) + sum(ctx)
    else:
        seen = sum(x * c for x, c in zip(new, ctx))
        keys = sum(ctx)
    return {"bytes": keys * (2 * H * (NOPE + DVX) + 2 * ROPE) + n * H * (2 * (NOPE + ROPE) + 2 * DVX + 4),
            "flops": 2.0 * H * (NOPE + ROPE + DVX) * seen}


# ---------------------------------------------------------------- the definition in 64 bits

def _row_of(s, b, t):
    return s.table[b, t // PAGE].long(), t % PAGE


def _attend(x, v, last):
    """out, lse of scores x [..., n, m] of which query i sees the first
    last[i] keys."""
    x = x.masked_fill(torch.arange(x.shape[-1], device=DEV) >= last[:, None], -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
    return p @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    at = s.starts.tolist()
    if case["op"] in ("append", "read"):
        pool = s.kv.view(torch.float8_e4m3fn).double() if case["kv"] == "e4m3" else s.kv.double()
        scale = float(s.divisor)
        if case["op"] == "read":
            out = torch.zeros(s.out.shape, dtype=torch.float64, device=DEV)
        for b, (n, c) in enumerate(zip(s.new, s.ctx)):
            page, r = _row_of(s, b, c + torch.arange(n, device=DEV))
            if case["op"] == "append":
                pool[page, r] = s.rows[at[b]:at[b] + n].double() / scale
            else:
                out[at[b]:at[b] + n] = pool[page, r] * scale
        return {"kv": pool} if case["op"] == "append" else {"rows": out}
    out = torch.zeros(s.out.shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s.lse.shape, dtype=torch.float64, device=DEV)
    for b, (n, c) in enumerate(zip(s.new, s.ctx)):
        if case["op"] == "chunk":
            kv = s.kv[_row_of(s, b, torch.arange(c + n, device=DEV))]
            kv = kv.view(torch.float8_e4m3fn).double() * float(s.divisor) if case["kv"] == "e4m3" else kv.double()
        else:
            first, m = int(s.k_starts[b]), s.keys[b]
            up = s.up[first:first + m].double()
            k = torch.cat([up[..., :NOPE], s.latent[first:first + m, None, DV:].double().expand(m, case["heads"], ROPE)],
                          -1).transpose(0, 1)
            v = up[..., NOPE:].transpose(0, 1)
        for i in range(0, n, 128):
            e = min(n, i + 128)
            q = s.q[at[b] + i:at[b] + e].double().transpose(0, 1)  # [H, tokens, dims]
            last = c + 1 + torch.arange(i, e, device=DEV)
            if case["op"] == "chunk":
                o, w = _attend(q @ kv.T / math.sqrt(192.0), kv[:, :DV], last)
            else:
                last = last if case["causal"] else torch.full_like(last, m)
                o, w = _attend(q @ k.transpose(1, 2) / math.sqrt(192.0), v, last)
            out[at[b] + i:at[b] + e] = o.transpose(0, 1)
            lse[at[b] + i:at[b] + e] = w.T
    return {"out": out, "lse": lse}
