"""Parallel samples of two prompts beside one long windowed conversation.

    python examples/parallel_samples.py [--steps 24] [--check]

A serving loop over one page pool: the prompts fork into samples that share
their full pages (pages_fork), every step reserves pages (pages_alloc), appends
the new token's latent row (kv_append) and decodes -- the samples with the
shared pages attended once per prompt (decode_shared), the conversation through
a sliding window with a few first tokens (decode_window), giving up the pages
behind the window (pages_free).  Half of the samples end early; their pages are
freed, the pool is compacted and the rest go on.  Queries and latent rows are
random: there is no model here, only its cache.  --check compares the last
step with the definition in 64 bits.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mla_paged_decode_gb300 as mla  # noqa: E402

PAGE, DQK, DV, HEADS = 64, 576, 512, 16
SCALE = 1.0 / math.sqrt(192.0)
WINDOW, SINKS = 256, 4
SAMPLES = 6          # of each prompt


def reference(q, kv, row, length, window=None):
    """out of one query at the last position, from the definition."""
    t = torch.arange(length, device=q.device)
    if window:
        t = t[(t > length - 1 - window) | (t < SINKS)]
    rows = kv[row[t // PAGE].long(), t % PAGE].double()
    p = torch.softmax(q.double() @ rows.T * SCALE, -1)
    return p @ rows[:, :DV]


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(0)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731

    # requests: 0 the conversation, 1 and 2 the prompts, then the samples
    prompts = [900, 517]
    first = 3
    rows, width, pages = first + 2 * SAMPLES, 32, 160
    kv = torch.zeros(pages, PAGE, DQK, dtype=torch.bfloat16, device=dev)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=dev)
    counts = torch.zeros(pages, dtype=torch.int32, device=dev)
    lens = torch.zeros(rows, dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ws = mla.make_pages_workspace(counts)

    # prefill: pages for the prompts, and what the model would write into them
    start = ints([700] + prompts + [0] * (2 * SAMPLES))
    mla.pages_alloc(table, lens, counts, start, workspace=ws, error_word=err)
    lens.copy_(start)
    for b in range(first):
        n = -(-int(start[b]) // PAGE)
        kv[table[b, :n].long()] = rnd(n, PAGE, DQK)

    # samples of a prompt sit next to each other: one group each
    samples = list(range(first, rows))
    mla.pages_fork(kv, table, lens, counts, ints([1] * SAMPLES + [2] * SAMPLES), ints(samples), workspace=ws,
                   error_word=err)
    group_starts = ints([0, SAMPLES, 2 * SAMPLES])
    shared = ints([n // PAGE for n in prompts])

    sample_table, sample_lens = table[first:], lens[first:]  # rows of the same storage
    q = rnd(2 * SAMPLES, 1, HEADS, DQK)
    out = torch.empty(2 * SAMPLES, 1, HEADS, DV, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(2 * SAMPLES, 1, HEADS, device=dev)
    cq, cout = rnd(1, 1, HEADS, DQK), torch.empty(1, 1, HEADS, DV, dtype=torch.bfloat16, device=dev)
    clse = torch.empty(1, 1, HEADS, device=dev)
    shared_ws = mla.make_shared_workspace(q, kv, sample_table, 2)
    window_ws = mla.make_workspace(cq, kv, table[:1])

    running = torch.ones(rows, dtype=torch.int32, device=dev)
    running[1:first] = 0                 # the prompts themselves do not grow
    for step in range(a.steps):
        if step == a.steps // 2:         # every other sample ends; close the gaps
            running[first::2] = 0
            ended = (torch.arange(rows, device=dev) >= first) & (running == 0)
            mla.pages_free(table, lens, counts, torch.where(ended, 0, lens), error_word=err)
            mla.pages_compact(kv, table, counts, workspace=ws, error_word=err)
        grown = lens + running
        mla.pages_alloc(table, lens, counts, grown, workspace=ws, error_word=err)
        mla.kv_append(rnd(rows, DQK), kv, table, torch.where(running > 0, lens, -1), error_word=err)
        lens.copy_(grown)
        mla.decode_shared(q, kv, sample_table, sample_lens, group_starts, shared, SCALE, mla.LSE_NATURAL, out, lse,
                          workspace=shared_ws)
        mla.decode_window(cq, kv, table[:1], lens[:1], WINDOW, SINKS, SCALE, mla.LSE_NATURAL, cout, clse,
                          workspace=window_ws)
        # pages behind the conversation's window go back to the pool
        mla.pages_free(table[:1], lens[:1], counts, lens[:1].clone(), window=WINDOW, sinks=SINKS, error_word=err)
    torch.cuda.synchronize()
    if int(err.item()) or mla.check_workspace(shared_ws) or mla.check_workspace(window_ws):
        raise SystemExit("a call reported an error")
    print(f"{a.steps} steps; lengths {lens.tolist()}; {int((counts > 0).sum())} of {pages} pages live")
    if a.check:
        worst = 0.0
        for i in range(2 * SAMPLES):
            if int(running[first + i]):
                want = reference(q[i, 0], kv, sample_table[i], int(sample_lens[i]))
                worst = max(worst, float((out[i, 0].double() - want).norm() / want.norm()))
        want = reference(cq[0, 0], kv, table[0], int(lens[0]), WINDOW)
        worst = max(worst, float((cout[0, 0].double() - want).norm() / want.norm()))
        print(f"largest relative error against 64 bits: {worst:.2e}")
        if not worst < 2.0**-7:          # weights and output rounded to bf16, half a step (2^-8) each
            raise SystemExit("the outputs are off")
    return 0


if __name__ == "__main__":
    sys.exit(main())
