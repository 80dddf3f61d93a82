"""Integer arguments that do not fit into the C calls' 32 bits are refused by
name, not cut to their low half (a window of 2**32 + 7 would become 7)."""
import pytest
import torch

import mla_paged_decode_gb300 as mla

q = torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16)
kv = torch.zeros(2, 64, 576, dtype=torch.bfloat16)
t = torch.zeros(1, 2, dtype=torch.int32)
one = torch.zeros(1, dtype=torch.int32)

CALLS = {
    "window": lambda v: mla.decode_window(q, kv, t, one, v, 0, 0.1, 0, q, q),
    "sinks": lambda v: mla.decode_window(q, kv, t, one, 8, v, 0.1, 0, q, q),
    "lse_base": lambda v: mla.decode_window(q, kv, t, one, 8, 0, 0.1, v, q, q),
    "lse_base (shared)": lambda v: mla.decode_shared(q, kv, t, one, t, one, 0.1, v, q, q),
    "window (free)": lambda v: mla.pages_free(t, one, one, one, window=v),
    "sinks (free)": lambda v: mla.pages_free(t, one, one, one, window=8, sinks=v),
    "num_pages": lambda v: mla.pages_workspace_size(v),
    "part_id": lambda v: mla.decode_partial(q, kv, t, one, v, 1, 0.1, 0, q, q),
    "num_parts": lambda v: mla.decode_partial(q, kv, t, one, 0, v, 0.1, 0, q, q),
    "num_parts (noalloc)": lambda v: mla.decode_partial_noalloc(q, kv, t, one, 0, v, 0.1, 0, q, q),
    "num_parts (dcp)": lambda v: mla.decode_dcp(q, kv, t, one, v, 0.1, 0),
    "num_parts (append)": lambda v: mla.kv_append(q[:, 0, 0], kv, t, one, 0, v),
    "num_parts (combine)": lambda v: mla.lse_combine(q, q, v, q),
    "max_pages": lambda v: mla.dcp_local_metadata(one, one, t, 0, 1, max_pages=v),
    "pad_value": lambda v: mla.dcp_local_metadata(one, one, t, 0, 1, max_pages=2, pad_value=v),
    "extra_tokens": lambda v: mla.dcp_local_metadata(one, one, t, 0, 1, max_pages=2, extra_tokens=v),
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("value", [2**32 + 7, 2**31, -2**31 - 1, -2**32])
def test_arguments_past_32_bits_are_refused(name, value):
    with pytest.raises(ValueError, match=rf"{name.split()[0]} = {value} does not fit into 32 bits"):
        CALLS[name](value)


def test_sizes_past_32_bits_are_refused():
    """(Sizes of tensors that take no memory.)"""
    wide = torch.zeros(1, dtype=torch.int32).expand(1, 2**31)
    with pytest.raises(ValueError, match="32 bits"):
        mla._make_decode_desc(q, kv, wide, 1.0)
    with pytest.raises(ValueError, match="32 bits"):
        mla._pages_desc(4, 2**32 + 8, 16, 64, 576, 0)
