"""Refusals of the chunk operators on the host: the C calls with bad arguments,
and the binding."""
import ctypes
import math

import pytest
import torch

import mla_paged_decode_gb300 as mla
from test_abi import FAKE, _desc, lib  # noqa: F401


def append(lib, d, *, rows=FAKE, stride=576, n=4, kv=FAKE, table=FAKE, starts=FAKE, pos=FAKE, part=0, parts=1, err=None):  # noqa: F811
    return lib.mla_kv_append_chunk(rows, stride, n, kv, table, starts, pos, part, parts,
                                   ctypes.byref(d) if d else None, err, None)


def read(lib, d, *, rows=FAKE, stride=576, n=4, kv=FAKE, table=FAKE, starts=FAKE, pos=FAKE, err=None):  # noqa: F811
    return lib.mla_kv_read(kv, table, starts, pos, rows, stride, n, ctypes.byref(d) if d else None, err, None)


def chunk(lib, d, *, n=4, scale=0.1, base=0, q=FAKE, kv=FAKE, table=FAKE, lens=FAKE, starts=FAKE, out=FAKE, lse=FAKE,  # noqa: F811
          ws=FAKE, size=1 << 40):
    return lib.mla_prefill_chunk(q, n, kv, table, lens, starts, scale, base, out, lse, ctypes.byref(d) if d else None,
                                 ws, size, None)


def edesc(**kw):
    base = dict(batch=2, num_heads=16, q_tokens=8, k_tokens=9, causal=1, q_token_stride=3200, q_head_stride=192,
                k_token_stride=4096, k_head_stride=256, rope_token_stride=576, v_token_stride=4096, v_head_stride=256)
    base.update(kw)
    return mla.ExpandedDesc(**base)


def expanded(lib, d, *, scale=0.1, base=0, q=FAKE, kn=FAKE, kr=FAKE, v=FAKE, qs=FAKE, ks=FAKE, out=FAKE, lse=FAKE,  # noqa: F811
             ws=FAKE, size=1 << 40):
    return lib.mla_prefill_expanded(q, kn, kr, v, qs, ks, scale, base, out, lse, ctypes.byref(d) if d else None, ws,
                                    size, None)


@pytest.mark.parametrize("call", [append, read])
def test_rows(lib, call):  # noqa: F811
    assert call(lib, None) == -1
    for kw, code in [(dict(page_size=32), -2), (dict(num_pages=0), -2), (dict(batch=-1), -2), (dict(kv_dtype=5), -6),
                     (dict(kv_dtype=1, kv_scale=0.0), -6), (dict(head_dim_qk=512), -2)]:
        assert call(lib, _desc(**kw)) == code, kw
    assert call(lib, _desc(), n=-1) == call(lib, _desc(), stride=575) == call(lib, _desc(), stride=-576) == -2
    assert call(lib, _desc(), stride=577) == -4
    for name in ("rows", "kv", "table", "starts", "pos"):
        assert call(lib, _desc(), **{name: None}) == -1, name
        assert call(lib, _desc(), **{name: FAKE + 2}) == -4, name
    assert call(lib, _desc(), rows=FAKE + 8) == call(lib, _desc(), err=FAKE + 1) == -4
    assert call(lib, _desc(batch=0), rows=None) == call(lib, _desc(), rows=None, n=0) == 0


def test_partitions(lib):  # noqa: F811
    assert append(lib, _desc(), part=2, parts=2) == append(lib, _desc(), part=-1) == append(lib, _desc(), parts=0) == -3


def test_chunk(lib):  # noqa: F811
    assert chunk(lib, None) == -1
    for kw, code in [(dict(num_heads=129), -2), (dict(num_heads=0), -2), (dict(page_size=32), -2), (dict(batch=-1), -2),
                     (dict(kv_dtype=5), -6), (dict(kv_dtype=1, kv_scale=math.nan), -6), (dict(head_dim_v=128), -2)]:
        assert chunk(lib, _desc(**kw)) == code, kw
    assert chunk(lib, _desc(), n=-1) == chunk(lib, _desc(), n=1 << 27) == -2
    assert chunk(lib, _desc(batch=(1 << 20) + 1)) == -2
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert chunk(lib, _desc(), scale=scale) == -6
    assert chunk(lib, _desc(), base=2) == -6
    for name in ("q", "kv", "table", "lens", "starts", "out", "lse", "ws"):
        assert chunk(lib, _desc(), **{name: None}) == -1, name
        assert chunk(lib, _desc(), **{name: FAKE + 2}) == -4, name
    assert chunk(lib, _desc(), ws=FAKE + 16) == -4
    assert chunk(lib, _desc(batch=0), q=None) == chunk(lib, _desc(), n=0, q=None) == 0


def test_expanded(lib):  # noqa: F811
    assert expanded(lib, None) == -1
    for kw, code in [(dict(num_heads=129), -2), (dict(num_heads=0), -2), (dict(batch=-1), -2), (dict(q_tokens=-1), -2),
                     (dict(k_tokens=-1), -2), (dict(k_tokens=(1 << 30) + 1), -2), (dict(q_tokens=1 << 27), -2),
                     (dict(batch=(1 << 20) + 1), -2), (dict(causal=2), -6)]:
        assert expanded(lib, edesc(**kw)) == code, kw
    for name in ("q_token_stride", "q_head_stride", "k_token_stride", "k_head_stride", "rope_token_stride",
                 "v_token_stride", "v_head_stride"):
        assert expanded(lib, edesc(**{name: 0})) == expanded(lib, edesc(**{name: -8})) == -2, name
        assert expanded(lib, edesc(**{name: 1 << 38})) == -2, name
        assert expanded(lib, edesc(**{name: 260})) == -4, name
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert expanded(lib, edesc(), scale=scale) == -6
    assert expanded(lib, edesc(), base=2) == -6
    for name in ("q", "kn", "kr", "v", "qs", "ks", "out", "lse", "ws"):
        assert expanded(lib, edesc(), **{name: None}) == -1, name
        assert expanded(lib, edesc(), **{name: FAKE + 2}) == -4, name
    assert expanded(lib, edesc(batch=0), q=None) == expanded(lib, edesc(q_tokens=0), q=None) == 0


def test_workspace_size(lib):  # noqa: F811
    # two slots of 512 rows of 128 + 1 floats a pair of SMs, and of 64 rows of 512 + 1 a SM
    assert lib.mla_prefill_workspace_size(152) >= max(152 * 512 * 129 * 4, 304 * 64 * 513 * 4)
    assert lib.mla_prefill_workspace_size(8) < lib.mla_prefill_workspace_size(152)


kv = torch.zeros(2, 64, 576, dtype=torch.bfloat16)
t = torch.zeros(1, 2, dtype=torch.int32)
one, two = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
rows = torch.zeros(3, 576, dtype=torch.bfloat16)
q, qx = torch.zeros(3, 16, 576, dtype=torch.bfloat16), torch.zeros(3, 16, 192, dtype=torch.bfloat16)
k = torch.zeros(4, 16, 128, dtype=torch.bfloat16)
lse = torch.zeros(3, 16)


def test_the_binding_refuses_cpu_tensors():
    for call in (lambda: mla.kv_append_chunk(rows, kv, t, two, one), lambda: mla.kv_read(kv, t, two, one, rows),
                 lambda: mla.prefill_chunk(q, kv, t, one, two, 0.1, 0, q, lse),
                 lambda: mla.prefill_expanded(qx, k, rows[:, :64], k, two, two, True, 0.1, 0, k, lse)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("value", [2**32 + 7, 2**31, -2**31 - 1])
def test_arguments_past_32_bits_are_refused(value):
    for name, call in {"part_id": lambda: mla.kv_append_chunk(rows, kv, t, two, one, value, 1),
                       "num_parts": lambda: mla.kv_append_chunk(rows, kv, t, two, one, 0, value),
                       "lse_base": lambda: mla.prefill_chunk(q, kv, t, one, two, 0.1, value, q, lse)}.items():
        with pytest.raises(ValueError, match=f"{name} = {value} does not fit into 32 bits"):
            call()
    with pytest.raises(ValueError, match="lse_base"):
        mla.prefill_expanded(qx, k, rows[:, :64], k, two, two, True, 0.1, value, k, lse)


def test_descriptor_checks():
    """The checks behind the device's: shapes and strides."""
    rope = rows[:, :64].expand(3, 64)
    ok = (qx, k[:3], rope, k[:3])
    mla._expanded_desc(*ok, 1, True)
    bad = [(qx[..., :128], *ok[1:]), (qx, k, *ok[2:]), (qx, k[:3, :8], *ok[2:]), (*ok[:3], k[:3, :, :64]),
           (qx, k[:3], rows, k[:3]), (qx.transpose(1, 2).contiguous().transpose(1, 2), *ok[1:]), (qx[0], *ok[1:])]
    for case in bad:
        with pytest.raises(ValueError):
            mla._expanded_desc(*case, 1, True)
    for i in range(4):
        for other in (ok[i].float(), None, ok[i].tolist()):
            with pytest.raises(TypeError):
                mla._expanded_desc(*ok[:i], other, *ok[i + 1:], 1, True)
    for case in ((kv[..., :512], t), (kv[0], t), (kv, one), (kv, t.expand(3, 2))):
        with pytest.raises(ValueError):
            mla._cache_desc(1, 16, *case, 1.0)
