"""Refusals of decode_window and decode_shared on the host, and the sizes of
their workspaces."""
import ctypes
import math

import pytest
import torch

import mla_paged_decode_gb300 as mla
from test_abi import FAKE, _desc, lib  # noqa: F401


def window(lib, d, *, window=8, sinks=0, scale=0.1, base=0, q=FAKE, kv=FAKE, out=FAKE, ws=FAKE, size=1 << 40):  # noqa: F811
    return lib.mla_decode_window(q, kv, FAKE, FAKE, window, sinks, scale, base, out, FAKE,
                                 ctypes.byref(d) if d else None, ws, size, None)


def shared(lib, d, *, groups=1, scale=0.1, base=0, q=FAKE, kv=FAKE, out=FAKE, ws=FAKE, size=1 << 40,  # noqa: F811
           starts=FAKE, pages=FAKE):
    return lib.mla_decode_shared(q, kv, FAKE, FAKE, starts, pages, groups, scale, base, out, FAKE,
                                 ctypes.byref(d) if d else None, ws, size, None)


@pytest.mark.parametrize("call", [window, shared])
@pytest.mark.parametrize("kw,code", [(dict(q_len=17), -2), (dict(num_heads=129), -2), (dict(page_size=32), -2),
                                     (dict(num_pages=0), -2), (dict(batch=-1), -2), (dict(kv_dtype=5), -6),
                                     (dict(kv_dtype=1, kv_scale=math.inf), -6),
                                     (dict(batch=1 << 30, num_heads=2), -2)])
def test_bad_descriptors(lib, call, kw, code):  # noqa: F811
    assert call(lib, _desc(**kw)) == code


@pytest.mark.parametrize("call", [window, shared])
def test_common_refusals(lib, call):  # noqa: F811
    assert call(lib, None) == -1
    assert call(lib, _desc(), base=2) == call(lib, _desc(), scale=math.nan) == -6
    assert call(lib, _desc(), scale=0.0) == call(lib, _desc(), scale=-1.0) == -6
    for name in ("q", "kv", "out", "ws"):
        assert call(lib, _desc(), **{name: None}) == -1, name
        assert call(lib, _desc(), **{name: FAKE + 8}) == -4, name
    assert call(lib, _desc(batch=0), q=None) == 0


def test_window_arguments(lib):  # noqa: F811
    assert window(lib, _desc(), window=0) == window(lib, _desc(), sinks=-1) == -6


def test_shared_arguments(lib):  # noqa: F811
    assert shared(lib, _desc(), groups=0) == shared(lib, _desc(), groups=(1 << 20) + 1) == -6
    assert shared(lib, _desc(), starts=None) == shared(lib, _desc(), pages=None) == -1
    assert shared(lib, _desc(), starts=FAKE + 2) == shared(lib, _desc(), pages=FAKE + 1) == -4


def test_shared_workspace_size(lib):  # noqa: F811
    size = lambda groups=1, **kw: lib.mla_decode_shared_workspace_size(ctypes.byref(_desc(**kw)), groups, 152)  # noqa: E731
    assert size(q_len=17) == size(groups=0) == 0
    # a slot of 64 x (512 + 1) floats for every virtual request and CTA
    assert size(batch=4, num_heads=64) >= (4 + 1 + 4 + 152) * 64 * 513 * 4
    assert size(groups=5) > size(groups=1)


def test_the_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16)
    kv = torch.zeros(2, 64, 576, dtype=torch.bfloat16)
    i = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.decode_window(q, kv, i, i[0, :1], 8, 0, 0.1, 0, q, q)
    with pytest.raises(ValueError):
        mla.decode_shared(q, kv, i, i[0, :1], i[0], i[0, :1], 0.1, 0, q, q)
