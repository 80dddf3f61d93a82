"""Prompts served in chunks over one paged latent cache, both ways.

    python examples/chunked_prefill.py [--chunk 200] [--check]

Three prompts of different lengths go through a layer chunk by chunk, a chunk of
each beside the others while it lasts.  Every step reserves pages
(pages_alloc), writes the chunk's latent rows into the cache
(kv_append_chunk) and attends to everything up to each token:

* absorbed: the queries multiplied by the key projection attend to the cache
  itself (prefill_chunk), and their outputs are multiplied by the value
  projection;
* expanded: the rows before the chunk are read back from the cache (kv_read),
  keys and values of all heads come from the two projections, the chunk attends
  to its own keys with a causal mask and to the earlier ones without
  (prefill_expanded), and both parts are merged (lse_combine).

The last step decodes one token of each (decode_partial).  Latent rows, queries
and projections are random: there is no model here, only its attention.
--check compares both ways with the definition in 64 bits.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mla_paged_decode_gb300 as mla  # noqa: E402

PAGE, LATENT, ROPE, NOPE, DV, HEADS = 64, 512, 64, 128, 128, 16
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
PROMPTS = [900, 517, 64]


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--chunk", type=int, default=200)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(0)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    starts_of = lambda n: ints([0] + n).cumsum(0).to(torch.int32)  # noqa: E731

    B = len(PROMPTS)
    kv = torch.zeros(60, PAGE, LATENT + ROPE, dtype=torch.bfloat16, device=dev)
    table = torch.full((B, 16), -1, dtype=torch.int32, device=dev)
    counts = torch.zeros(60, dtype=torch.int32, device=dev)
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    pages_ws = mla.make_pages_workspace(counts)
    w_k = rnd(HEADS, NOPE, LATENT) * LATENT**-0.5      # a head's keys and values from the latent
    w_v = rnd(HEADS, DV, LATENT) * LATENT**-0.5
    w_up = torch.cat([w_k, w_v], 1).view(-1, LATENT)
    rows = [rnd(n + 1, LATENT + ROPE) for n in PROMPTS]
    queries = [rnd(n + 1, HEADS, NOPE + ROPE) for n in PROMPTS]
    workspace = mla.make_prefill_workspace(kv)
    worst = {"absorbed": 0.0, "expanded": 0.0}

    def definition(b, first, n):
        """out of request b's queries first .. first + n, in 64 bits."""
        q, x = queries[b][first:first + n].double(), rows[b][:first + n].double()
        k = torch.einsum("td,hkd->thk", x[:, :LATENT], w_k.double())
        s = torch.einsum("nhk,thk->nht", q[..., :NOPE], k) + torch.einsum("nhk,tk->nht", q[..., NOPE:], x[:, LATENT:])
        t = torch.arange(first + n, device=dev)
        s = (s * SCALE).masked_fill((t > first + torch.arange(n, device=dev)[:, None])[:, None], -math.inf)
        return torch.einsum("nht,td,hkd->nhk", torch.softmax(s, -1), x[:, :LATENT], w_v.double())

    done = [0] * B
    while any(d < n for d, n in zip(done, PROMPTS)):
        new = [min(a.chunk, n - d) for d, n in zip(done, PROMPTS)]
        N, starts, before = sum(new), starts_of(new), ints(done)
        grown = lens + ints(new)
        chunk_rows = torch.cat([r[d:d + n] for r, d, n in zip(rows, done, new)])
        q = torch.cat([x[d:d + n] for x, d, n in zip(queries, done, new)])
        mla.pages_alloc(table, lens, counts, grown, workspace=pages_ws, error_word=err)
        mla.kv_append_chunk(chunk_rows, kv, table, starts, before, error_word=err)
        lens.copy_(grown)

        # absorbed: over the cache
        q_abs = torch.cat([torch.einsum("nhk,hkd->nhd", q[..., :NOPE], w_k), q[..., NOPE:]], -1)
        o_lat = torch.empty(N, HEADS, LATENT, dtype=torch.bfloat16, device=dev)
        lse = torch.empty(N, HEADS, device=dev)
        mla.prefill_chunk(q_abs, kv, table, lens, starts, SCALE, mla.LSE_NATURAL, o_lat, lse, workspace=workspace)
        absorbed = torch.einsum("nhd,hkd->nhk", o_lat, w_v)

        # expanded: the chunk's own keys, and the cached rows before them
        parts = torch.empty(2, N, HEADS, DV, dtype=torch.bfloat16, device=dev)
        lses = torch.empty(2, N, HEADS, device=dev)
        context = torch.empty(sum(done), LATENT + ROPE, dtype=torch.bfloat16, device=dev)
        context_starts = starts_of(done)
        mla.kv_read(kv, table, context_starts, torch.zeros_like(lens), context, error_word=err)
        for part, (x, k_starts) in enumerate([(chunk_rows, starts), (context, context_starts)]):
            up = (x[:, :LATENT] @ w_up.T).view(-1, HEADS, NOPE + DV)
            mla.prefill_expanded(q, up[..., :NOPE], x[:, LATENT:], up[..., NOPE:], starts, k_starts, part == 0, SCALE,
                                 mla.LSE_NATURAL, parts[part], lses[part], workspace=workspace)
        expanded = torch.empty(N, HEADS, DV, dtype=torch.bfloat16, device=dev)
        mla.lse_combine(parts, lses, 2, expanded)

        if a.check:
            want = torch.cat([definition(b, d, n) for b, (d, n) in enumerate(zip(done, new)) if n])
            for name, got in (("absorbed", absorbed), ("expanded", expanded)):
                worst[name] = max(worst[name], float((got.double() - want).norm() / want.norm()))
        done = [d + n for d, n in zip(done, new)]

    # one token of each request
    grown = lens + 1
    mla.pages_alloc(table, lens, counts, grown, workspace=pages_ws, error_word=err)
    mla.kv_append(torch.stack([r[-1] for r in rows]), kv, table, lens, error_word=err)
    lens.copy_(grown)
    q = torch.stack([x[-1] for x in queries])[:, None]
    q_abs = torch.cat([torch.einsum("bthk,hkd->bthd", q[..., :NOPE], w_k), q[..., NOPE:]], -1)
    o_lat = torch.empty(B, 1, HEADS, LATENT, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(B, 1, HEADS, device=dev)
    mla.decode_partial(q_abs, kv, table, lens, 0, 1, SCALE, mla.LSE_NATURAL, o_lat, lse)
    torch.cuda.synchronize()
    if int(err.item()) or mla.check_workspace(workspace):
        raise SystemExit("a call reported an error")
    print(f"lengths {lens.tolist()}; {int((counts > 0).sum())} pages live")
    if a.check:
        print("largest relative error against 64 bits: " + ", ".join(f"{k} {v:.2e}" for k, v in worst.items()))
        # bf16 roundings of half a step, 2^-8, one after the other, in a 2-norm: projected
        # queries or keys and values, weights, parts, outputs, projected outputs
        if not max(worst.values()) < 5 * 2.0**-8:
            raise SystemExit("the outputs are off")
    return 0


if __name__ == "__main__":
    sys.exit(main())
