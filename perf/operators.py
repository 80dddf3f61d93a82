"""Cases of the shared-prefix decode, the windowed decode and the page operations.

Each case runs one pass of one operator on a paged latent cache (pages of 64
rows of 576 values): with ``own`` true through the library's calls, otherwise
in plain torch operations in fp32.  ``exact`` is the attention's definition in
64 bits; the page operations move bits and whole numbers, which have no
rounded value.
"""
import math

import torch

own = False

PAGE, DQK, DV = 64, 576, 512
SM_SCALE = 1.0 / math.sqrt(192.0)
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a few samples of one short prompt: latency
        dict(name="shared_small", op="shared", heads=16, q_len=1, kv="bf16", groups=1, per_group=4,
             prefix_pages=8, tail=48, ragged=False),
        # three prompts of a batch with different numbers of samples, two
        # draft tokens each, e4m3 cache, all heads on one GPU
        dict(name="shared_groups_e4m3", op="shared", heads=128, q_len=2, kv="e4m3", groups=3,
             per_group=13, prefix_pages=131, tail=700, ragged=True),
        # a batch of 64 over one 32K-token document
        dict(name="shared_32k", op="shared", heads=64, q_len=1, kv="bf16", groups=1, per_group=64,
             prefix_pages=512, tail=1500, ragged=True),
        # one short conversation under a small window: latency
        dict(name="window_small", op="window", heads=16, q_len=1, kv="bf16", batch=1, len_lo=300,
             len_hi=300, window=128, sinks=4),
        # the 4K..32K batch of 64 with 64 heads, the last 4096 tokens and 4 sinks
        dict(name="window_4k", op="window", heads=64, q_len=1, kv="bf16", batch=64, len_lo=4096,
             len_hi=32768, window=4096, sinks=4),
        # three tokens to verify for each request, e4m3 cache, odd window
        dict(name="window_mtp_e4m3", op="window", heads=128, q_len=3, kv="e4m3", batch=32, len_lo=1024,
             len_hi=16384, window=1999, sinks=70),
        # two requests branch into four samples each
        dict(name="fork_small", op="fork", kv="bf16", rows=16, parents=2, children=8, len_hi=1000,
             pages=512),
        # a beam step: 500 parents of up to 8K tokens branch into 1500 children
        dict(name="fork_beams", op="fork", kv="bf16", rows=2048, parents=500, children=1500,
             len_hi=8192, pages=17000),
        # a handful of finished requests leave a small pool
        dict(name="reclaim_small", op="reclaim", kv="bf16", rows=24, len_hi=1500, pages=600, drop=0.4),
        # a third of a large batch finishes, the rest is trimmed or kept
        dict(name="reclaim_large", op="reclaim", kv="bf16", rows=400, len_hi=4096, pages=14001, drop=0.35),
        # one request's pages go to another pool
        dict(name="copy_small", op="copy", kv="bf16", pages=300, moved=5),
        # a third of a pool goes to another pool, e4m3 rows
        dict(name="copy_large", op="copy", kv="e4m3", pages=30000, moved=10007),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "window", "window", "fork", "reclaim", "copy"])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    if op == "shared":
        while True:
            c = dict(op=op, heads=rng.choice([16, 64, 128, rng.randint(1, 128)]),
                     q_len=rng.choice([1, 1, 1, rng.randint(2, 4)]), kv=kv, groups=rng.choice([1, 1, 2, 3]),
                     per_group=_log_int(rng, 2, 64), prefix_pages=_log_int(rng, 4, 512),
                     tail=_log_int(rng, 1, 1500), ragged=rng.random() < 0.7)
            batch = c["groups"] * c["per_group"]
            tokens = 64 * c["prefix_pages"] + c["tail"]
            # no more work or temporaries than the 32K batch
            if (batch * c["heads"] * c["q_len"] * tokens <= 64 * 64 * (64 * 512 + 1500)
                    and batch * tokens <= 64 * (64 * 512 + 1500)):
                return c
    if op == "window":
        while True:
            hi = _log_int(rng, 64, 32768)
            c = dict(op=op, heads=rng.choice([16, 64, 128, rng.randint(1, 128)]),
                     q_len=rng.choice([1, 1, 1, rng.randint(2, 4)]), kv=kv, batch=_log_int(rng, 1, 64),
                     len_lo=rng.randint(1, hi), len_hi=hi, window=_log_int(rng, 32, 4096),
                     sinks=rng.choice([0, 1, 4, 16, rng.randint(0, 256)]))
            seen = min(hi, c["window"] + c["sinks"])
            if c["batch"] * c["heads"] * c["q_len"] * seen <= 64 * 64 * 4100:
                return c
    if op == "fork":
        parents = _log_int(rng, 1, 500)
        children = _log_int(rng, parents, min(1500, 8 * parents + 8))
        hi = _log_int(rng, 70, 8192)
        pages = min(17000, parents * (-(-hi // PAGE)) // 2 + children + rng.randint(64, 400))
        return dict(op=op, kv=kv, rows=parents + children + rng.randint(0, 40), parents=parents,
                    children=children, len_hi=hi, pages=pages)
    if op == "reclaim":
        rows = _log_int(rng, 4, 400)
        hi = _log_int(rng, 64, 4096)
        return dict(op=op, kv=kv, rows=rows, len_hi=hi,
                    pages=min(14001, rows * (-(-hi // PAGE)) // 2 + rng.randint(70, 300)),
                    drop=round(rng.uniform(0.1, 0.9), 3))
    pages = _log_int(rng, 64, 15000 if kv == "bf16" else 30000)
    return dict(op=op, kv=kv, pages=pages, moved=max(1, int(pages * rng.uniform(0.02, 0.33))))


# ---------------------------------------------------------------- inputs

class State:
    """What a serving loop holds: the pool, its tables and the call's buffers."""


def _generators(seed):
    c, g = torch.Generator(), torch.Generator(device=DEV)
    c.manual_seed(seed * 7919 + 11)
    g.manual_seed(seed * 104729 + 13)
    return c, g


def _pool(pages, kv, gen):
    """A latent cache of N(0, 1) rows: bf16, or e4m3 codes with one scale."""
    x = torch.empty(pages, PAGE, DQK, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=gen)
    if kv == "bf16":
        return x, 1.0
    scale = 5.5 / 448.0
    return (x.float() / scale).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _lens(case, gen):
    """Global lengths of an attention case, on the host."""
    if case["op"] == "window":
        n = torch.randint(case["len_lo"], case["len_hi"] + 1, (case["batch"],), generator=gen)
        return n.tolist()
    n = case["groups"] * case["per_group"]
    tail = torch.randint(1, case["tail"] + 1, (n,), generator=gen) if case["ragged"] else \
        torch.full((n,), case["tail"])
    pages = torch.tensor(_prefix(case)).repeat_interleave(case["per_group"])
    # the last q_len tokens of a request are its own
    return (64 * pages + tail.clamp(min=case["q_len"])).tolist()


def _prefix(case):
    """Shared pages of each group: the first has prefix_pages, later ones fewer."""
    return [max(1, case["prefix_pages"] - g * (case["prefix_pages"] // 5)) for g in range(case["groups"])]


def _prepare_attention(case, seed, s):
    cpu, gen = _generators(seed)
    lens = _lens(case, cpu)
    need = [-(-n // PAGE) for n in lens]
    width = max(need)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    if case["op"] == "shared":
        sp = _prefix(case)
        per = case["per_group"]
        total = sum(sp) + sum(n - sp[b // per] for b, n in enumerate(need))
        perm = torch.randperm(total, generator=cpu).to(torch.int32)
        at = 0
        for g, k in enumerate(sp):
            table[g * per:(g + 1) * per, :k] = perm[at:at + k]
            at += k
        for b, n in enumerate(need):
            k = sp[b // per]
            table[b, k:n] = perm[at:at + n - k]
            at += n - k
        s.group_starts = torch.arange(0, len(lens) + 1, per, dtype=torch.int32).to(DEV)
        s.shared_pages = torch.tensor(sp, dtype=torch.int32).to(DEV)
    else:
        total = sum(need)
        perm = torch.randperm(total, generator=cpu).to(torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
    s.kv, s.scale = _pool(total, case["kv"], gen)
    s.table = table.to(DEV)
    s.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    rows = (len(lens), case["q_len"], case["heads"])
    s.q = torch.randn(*rows, DQK, generator=gen, device=DEV).to(torch.bfloat16)
    s.out = torch.empty(*rows, DV, dtype=torch.bfloat16, device=DEV)
    s.lse = torch.empty(*rows, dtype=torch.float32, device=DEV)
    s.workspace = None


def _page_lens(case, gen):
    """Lengths of the requests a page case starts with: spread over (0, len_hi],
    as many as its pages hold."""
    n = case["parents"] if case["op"] == "fork" else case["rows"]
    lens = torch.randint(1, case["len_hi"] + 1, (n,), generator=gen).tolist()
    spare = case["children"] if case["op"] == "fork" else case["pages"] // 16
    left, got = case["pages"] - spare, []
    for x in lens:
        x = min(x, max(0, left) * PAGE)
        got.append(x)
        left -= -(-x // PAGE)
    return got


def _prepare_pages(case, seed, s):
    cpu, gen = _generators(seed)
    s.kv, _ = _pool(case["pages"], case["kv"], gen)
    if case["op"] == "copy":
        s.other, _ = _pool(case["pages"], case["kv"], gen)
        s.src = torch.randperm(case["pages"], generator=cpu)[:case["moved"]].to(torch.int32).to(DEV)
        s.dst = torch.randperm(case["pages"], generator=cpu)[:case["moved"]].to(torch.int32).to(DEV)
        return
    lens = _page_lens(case, cpu)
    rows, width = case["rows"], -(-case["len_hi"] // PAGE)
    perm = torch.randperm(case["pages"], generator=cpu).to(torch.int32)
    table = torch.full((rows, width), -1, dtype=torch.int32)
    counts = torch.zeros(case["pages"], dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // PAGE)
        table[b, :k] = perm[at:at + k]
        at += k
    counts[perm[:at].long()] = 1
    full = torch.zeros(rows, dtype=torch.int32)
    full[:len(lens)] = torch.tensor(lens, dtype=torch.int32)
    # the metadata as one buffer: a step works on a copy of the last committed one
    s.committed = torch.cat([table.flatten(), full, counts]).to(DEV)
    s.meta = s.committed.clone()
    s.table, s.lens, s.counts = _meta(s.meta, rows, width)
    if case["op"] == "fork":
        n = case["parents"]
        s.parents = torch.randint(0, n, (case["children"],), generator=cpu).to(torch.int32).to(DEV)
        s.children = (n + torch.randperm(rows - n, generator=cpu)[:case["children"]]).to(torch.int32).to(DEV)
    else:
        gone = torch.rand(rows, generator=cpu) < case["drop"]
        cut = torch.rand(rows, generator=cpu) < 0.25
        keep = torch.where(cut, (full * torch.rand(rows, generator=cpu)).to(torch.int32), full)
        s.new_lens = torch.where(gone, torch.zeros_like(full), keep).to(DEV)
        s.remap = torch.empty(case["pages"], dtype=torch.int32, device=DEV)
    s.workspace = None


def _meta(flat, rows, width):
    return flat[:rows * width].view(rows, width), flat[rows * width:rows * width + rows], \
        flat[rows * width + rows:]


def prepare(case, seed):
    s = State()
    s.case = case
    (_prepare_attention if case["op"] in ("shared", "window") else _prepare_pages)(case, seed, s)
    if own:
        import mla_paged_decode_gb300 as mla
        s.mla = mla
        if case["op"] == "shared":
            s.workspace = mla.make_shared_workspace(s.q, s.kv, s.table, case["groups"], s.scale)
        elif case["op"] == "window":
            s.workspace = mla.make_workspace(s.q, s.kv, s.table, s.scale)
        elif case["op"] != "copy":
            s.workspace = mla.make_pages_workspace(s.counts)
    return s


# ---------------------------------------------------------------- plain forms

def _rows(s, pages):
    """fp32 rows of the listed pages."""
    x = s.kv[pages]
    if s.case["kv"] == "e4m3":
        return x.view(torch.float8_e4m3fn).float() * s.scale
    return x.float()


def _attend(s, kv, seen):
    """out, lse of q over kv [B, N, 576] where seen [B, T, N]."""
    B, T, H, _ = s.q.shape
    q = s.q.float().view(B, T * H, DQK)
    x = torch.bmm(q, kv.transpose(1, 2)).view(B, T, H, -1) * SM_SCALE
    x = x.masked_fill(~seen[:, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = torch.bmm(p.view(B, T * H, -1), kv[..., :DV]).view(B, T, H, DV)
    lse = (top + torch.log(total)).squeeze(-1)
    return out.to(torch.bfloat16), lse


def _plain_shared(s):
    B, T = s.q.shape[:2]
    width = s.table.shape[1]
    kv = _rows(s, s.table.clamp(min=0).long()).view(B, width * PAGE, DQK)
    t = torch.arange(width * PAGE, device=DEV)
    last = s.lens[:, None] - T + torch.arange(T, device=DEV)  # each query token's position
    return _attend(s, kv, t <= last[..., None])


def _plain_window(s):
    c = s.case
    B, T = s.q.shape[:2]
    W, S = c["window"], c["sinks"]
    width = s.table.shape[1]
    lens = s.lens.long()
    first = lens - T + 1 - W  # first token the first query token's window holds
    sink_pages = min(width, -(-S // PAGE))
    start = torch.clamp(first, min=0) // PAGE
    n_win = min(width, -(-(W + T - 1) // PAGE) + 1)
    win = start[:, None] + torch.arange(n_win, device=DEV)
    sink = torch.arange(sink_pages, device=DEV).expand(B, sink_pages)
    lp = torch.cat([sink, win], 1)
    # a window page that is also a sink page counts once
    valid = torch.cat([torch.ones_like(sink, dtype=torch.bool), win >= sink_pages], 1) & (lp < width)
    lp = lp.clamp(max=width - 1)
    pages = torch.gather(s.table.long(), 1, lp)
    kv = _rows(s, pages.clamp(min=0)).view(B, -1, DQK)
    t = (lp[..., None] * PAGE + torch.arange(PAGE, device=DEV)).view(B, 1, -1)
    pos = (lens[:, None] - T + torch.arange(T, device=DEV))[..., None]
    seen = (t <= pos) & ((t > pos - W) | (t < S)) & valid.repeat_interleave(PAGE, 1)[:, None]
    return _attend(s, kv, seen)


def _plain_fork(s):
    par, chi = s.parents.long(), s.children.long()
    L = s.lens[par]
    full, rem = (L // PAGE).long(), L % PAGE
    rows = s.table[par]
    col = torch.arange(rows.shape[1], device=DEV)
    held = (col < full[:, None]) & (rows >= 0)
    part = rem > 0
    free = torch.nonzero(s.counts == 0).flatten()
    new = free[:int(part.sum())]  # the lowest free pages, in the forks' order
    s.counts.index_add_(0, rows[held].long(), torch.ones_like(rows[held]))
    s.counts[new] = 1
    child = torch.where(held, rows, torch.full_like(rows, -1))
    k = torch.nonzero(part).flatten()
    old = rows[k, full[k]].long()
    child[k, full[k]] = new.to(torch.int32)
    s.table[chi] = child
    s.lens[chi] = L
    used = torch.arange(PAGE, device=DEV) < rem[k][:, None]
    s.kv[new] = torch.where(used[..., None], s.kv[old], s.kv[new])


def _plain_reclaim(s):
    width = s.table.shape[1]
    keep = torch.arange(width, device=DEV) < ((s.new_lens + PAGE - 1) // PAGE)[:, None]
    gone = ~keep & (s.table >= 0)
    ids = s.table[gone].long()
    s.counts.index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    s.table[gone] = -1
    s.lens.copy_(s.new_lens)
    live = s.counts > 0
    n = int(live.sum())
    holes = torch.nonzero(~live[:n]).flatten()
    movers = torch.nonzero(live[n:]).flatten() + n
    s.kv[holes] = s.kv[movers]
    s.counts[holes] = s.counts[movers]
    s.counts[movers] = 0
    s.remap.copy_(torch.where(live, torch.arange(live.numel(), device=DEV), -1))
    s.remap[movers] = holes.to(torch.int32)
    s.table.copy_(torch.where(s.table >= 0, s.remap[s.table.clamp(min=0).long()], s.table))


# ---------------------------------------------------------------- one pass

def run(s):
    op = s.case["op"]
    if op in ("shared", "window"):
        if not own:
            out, lse = (_plain_shared if op == "shared" else _plain_window)(s)
            return {"out": out, "lse": lse}
        if op == "shared":
            s.mla.decode_shared(s.q, s.kv, s.table, s.lens, s.group_starts, s.shared_pages, SM_SCALE,
                                s.mla.LSE_NATURAL, s.out, s.lse, kv_scale=s.scale, workspace=s.workspace)
        else:
            s.mla.decode_window(s.q, s.kv, s.table, s.lens, s.case["window"], s.case["sinks"], SM_SCALE,
                                s.mla.LSE_NATURAL, s.out, s.lse, kv_scale=s.scale, workspace=s.workspace)
        return {"out": s.out, "lse": s.lse}
    if op == "copy":
        if own:
            s.mla.pages_copy(s.kv, s.other, s.src, s.dst)
        else:
            s.other[s.dst.long()] = s.kv[s.src.long()]
        return {"kv": _words(s.other)}
    s.meta.copy_(s.committed)
    if op == "fork":
        if own:
            s.mla.pages_fork(s.kv, s.table, s.lens, s.counts, s.parents, s.children, workspace=s.workspace)
        else:
            _plain_fork(s)
        return {"kv": _words(s.kv), "table": s.table, "lens": s.lens, "counts": s.counts}
    if own:
        s.mla.pages_free(s.table, s.lens, s.counts, s.new_lens)
        s.mla.pages_compact(s.kv, s.table, s.counts, remap=s.remap, workspace=s.workspace)
    else:
        _plain_reclaim(s)
    return {"kv": _words(s.kv), "table": s.table, "lens": s.lens, "counts": s.counts, "remap": s.remap}


def _words(pool):
    """A pool as the 32-bit words that the page operations move, whatever they
    stand for: compared bit for bit."""
    return pool.view(torch.int32)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    row = DQK * (2 if case["kv"] == "bf16" else 1)
    if case["op"] in ("shared", "window"):
        if case["op"] == "shared":
            batch = case["groups"] * case["per_group"]
            tail = max(case["q_len"], (1 + case["tail"]) / 2 if case["ragged"] else case["tail"])
            sp = _prefix(case)
            kv_rows = PAGE * sum(sp) + batch * tail
            seen = PAGE * sum(sp) * case["per_group"] + batch * tail
        else:
            batch = case["batch"]
            n = (case["len_lo"] + case["len_hi"]) / 2
            kv_rows = batch * min(n, case["window"] + case["q_len"] - 1 + case["sinks"])
            seen = batch * min(n, case["window"] + case["sinks"])
        q_rows = batch * case["q_len"] * case["heads"]
        return {"bytes": kv_rows * row + q_rows * (2 * DQK + 2 * DV + 4),
                "flops": 2.0 * seen * case["q_len"] * case["heads"] * (DQK + DV)}
    if case["op"] == "copy":
        return {"bytes": 2.0 * case["moved"] * PAGE * row + 8 * case["moved"], "flops": 0}
    gen = torch.Generator()
    gen.manual_seed(5)
    lens = _page_lens(case, gen)
    n, width = max(1, len(lens)), -(-case["len_hi"] // PAGE)
    if case["op"] == "fork":
        mean_rows = sum(x % PAGE for x in lens) / n
        mean_pages = sum(-(-x // PAGE) for x in lens) / n
        return {"bytes": case["children"] * (2.0 * mean_rows * row + 4 * (mean_pages + width + 4))
                + 4 * case["pages"], "flops": 0}
    held = sum(-(-x // PAGE) for x in lens)
    kept = held * (1 - case["drop"]) * 0.875
    moved = kept * (1 - kept / case["pages"])
    return {"bytes": 2.0 * moved * PAGE * row + 8 * case["pages"] + 8 * case["rows"] * width, "flops": 0}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    if case["op"] not in ("shared", "window"):
        return None  # words moved and whole numbers: no rounded value
    s = State()
    s.case = case
    _prepare_attention(case, seed, s)
    B, T, H, _ = s.q.shape
    out = torch.zeros(B, T, H, DV, dtype=torch.float64, device=DEV)
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s.lens.tolist()):
        for i in range(T):
            pos = n - T + i
            t = torch.arange(0, max(0, pos + 1), device=DEV)
            if case["op"] == "window":
                t = t[(t > pos - case["window"]) | (t < case["sinks"])]
            if t.numel() == 0:
                continue
            page = s.table[b, t // PAGE].long()
            rows = s.kv[page, t % PAGE]
            rows = rows.view(torch.float8_e4m3fn).double() * s.scale if case["kv"] == "e4m3" else rows.double()
            x = s.q[b, i].double() @ rows.T / math.sqrt(192.0)
            lse[b, i] = torch.logsumexp(x, -1)
            out[b, i] = torch.softmax(x, -1) @ rows[:, :DV]
    return {"out": out, "lse": lse}
