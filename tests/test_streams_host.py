"""Scratch that the binding allocates for a call on a given stream comes from
that stream's pool: seen on the CPU with a stand-in for the stream's context."""
import contextlib

import pytest
import torch

import mla_paged_decode_gb300 as mla


class Stream:
    cuda_stream = 9


@pytest.fixture
def seen(monkeypatch):
    """Which context each workspace is made in ("current" or the stream's)."""
    made, inside = [], ["current"]

    @contextlib.contextmanager
    def on(stream):
        inside.append(stream)
        yield
        inside.pop()

    def make(*a, **k):
        made.append(inside[-1])
        return torch.zeros(256, dtype=torch.uint8)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: f"stream {ptr}")
    monkeypatch.setattr(mla, "_raw_stream", lambda index: 7)
    for name in ("make_workspace", "make_shared_workspace", "make_pages_workspace"):
        monkeypatch.setattr(mla, name, make)
    monkeypatch.setattr(mla, "_launch", lambda *a: None)
    monkeypatch.setattr(mla, "_view_args", lambda what, q, *a: (q.device, mla.DecodeDesc()))
    monkeypatch.setattr(mla, "_books", lambda dev, table, lens, counts, err: (*table.shape, counts.numel()))
    monkeypatch.setattr(mla, "_pool", lambda kv, name="": (kv.device, kv.shape, 0))
    return made


q = kv = torch.zeros(4, 64, 576, dtype=torch.bfloat16)
table = torch.zeros(2, 2, dtype=torch.int32)
one = torch.zeros(1, dtype=torch.int32)
two = torch.zeros(2, dtype=torch.int32)
four = torch.zeros(4, dtype=torch.int32)
CALLS = {
    "window": lambda **k: mla.decode_window(q, kv, table, two, 8, 0, 0.1, 0, q, q, **k),
    "shared": lambda **k: mla.decode_shared(q, kv, table, two, two, one, 0.1, 0, q, q, **k),
    "fork": lambda **k: mla.pages_fork(kv, table, two, four, one, one, **k),
    "alloc": lambda **k: mla.pages_alloc(table, two, four, two, **k),
    "compact": lambda **k: mla.pages_compact(kv, table, four, **k),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_default_scratch_belongs_to_the_given_stream(seen, name):
    CALLS[name](stream=Stream())
    CALLS[name]()
    assert seen == ["stream 9", "current"]
    Stream.cuda_stream, keep = 7, Stream.cuda_stream    # the current stream, given
    try:
        CALLS[name](stream=Stream())
    finally:
        Stream.cuda_stream = keep
    assert seen[2:] == ["current"]
