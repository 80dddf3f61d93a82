"""Refusals of the page operations, all on the host: no GPU and no memory is
touched by any of these calls."""
import ctypes

import pytest
import torch

import mla_paged_decode_gb300 as mla
from test_abi import FAKE, lib  # noqa: F401


def desc(**kw):
    base = dict(num_requests=4, max_pages_per_seq=8, num_pages=16, page_size=64, head_dim_qk=576, kv_dtype=0)
    base.update(kw)
    return ctypes.byref(mla.PagesDesc(**base))


def calls(lib, d, *, kv=FAKE, table=FAKE, lens=FAKE, counts=FAKE, lst=FAKE, ws=FAKE, ws_bytes=1 << 40,  # noqa: F811
          n=2, window=0, sinks=0, err=None):
    return {
        "copy": lib.mla_pages_copy(kv, FAKE, lst, FAKE, n, 9, d, err, None),
        "fork": lib.mla_pages_fork(kv, table, lens, counts, lst, FAKE, n, d, ws, ws_bytes, err, None),
        "alloc": lib.mla_pages_alloc(table, lens, counts, lst, d, ws, ws_bytes, err, None),
        "free": lib.mla_pages_free(table, lens, counts, lst, window, sinks, d, err, None),
        "compact": lib.mla_pages_compact(kv, table, counts, None, d, ws, ws_bytes, err, None),
    }


@pytest.mark.parametrize("kw,code", [
    (dict(num_requests=-1), -2), (dict(max_pages_per_seq=0), -2), (dict(num_pages=0), -2),
    (dict(page_size=32), -2), (dict(head_dim_qk=512), -2), (dict(kv_dtype=2), -6)])
def test_bad_descriptors(lib, kw, code):  # noqa: F811
    assert set(calls(lib, desc(**kw)).values()) == {code}


def test_null_and_misaligned_pointers(lib):  # noqa: F811
    assert set(calls(lib, None).values()) == {-1}
    for name, hit in (("kv", {"copy", "fork", "compact"}), ("table", {"fork", "alloc", "free", "compact"}),
                      ("lens", {"fork", "alloc", "free"}), ("lst", {"copy", "fork", "alloc", "free"}),
                      ("counts", {"fork", "alloc", "free", "compact"}), ("ws", {"fork", "alloc", "compact"})):
        got = calls(lib, desc(), **{name: None})
        assert {k for k, v in got.items() if v == -1} >= hit, name
        got = calls(lib, desc(), **{name: FAKE + 2})
        assert {k for k, v in got.items() if v == -4} >= hit, name
    assert set(calls(lib, desc(), err=FAKE + 1).values()) == {-4}


def test_bad_arguments(lib):  # noqa: F811
    got = calls(lib, desc(), n=-1)
    assert got["copy"] == got["fork"] == -6
    assert calls(lib, desc(), n=(1 << 19) + 1)["fork"] == -6
    assert calls(lib, desc(), window=-1)["free"] == calls(lib, desc(), sinks=-1)["free"] == -6
    assert lib.mla_pages_copy(FAKE, FAKE, FAKE, FAKE, 1, 0, desc(), None, None) == -2
    short = mla.pages_workspace_size(16) - 1
    got = calls(lib, desc(), ws_bytes=short)
    assert got["fork"] == got["alloc"] == got["compact"] == -5
    assert lib.mla_pages_workspace_size(0) == 0
    assert calls(lib, desc(num_requests=0), n=0)["fork"] == 0


def test_the_binding_refuses_cpu_tensors():
    t = torch.zeros(4, 8, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.pages_free(t, t[:, 0].contiguous(), torch.zeros(16, dtype=torch.int32), t[:, 0].contiguous())
    with pytest.raises(ValueError):
        mla.pages_copy(torch.zeros(4, 64, 576, dtype=torch.bfloat16),
                       torch.zeros(4, 64, 576, dtype=torch.bfloat16), t[0], t[0])
