"""Python binding of the GB300 MLA paged-decode C ABI (include/mla_decode.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``_lib/libmla_decode.so``.  PyTorch supplies device memory and the
current stream (or the `stream` given to a call, which then also owns the
workspace and outputs that the call allocates; the inputs have to be ready on
it).  If the library is not built, every call raises: there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

__all__ = [
    "MlaError", "LSE_NATURAL", "LSE_BASE2", "decode_partial", "lse_combine",
    "workspace_size", "make_workspace", "check_workspace", "library_path", "load_library",
    "decode_partial_noalloc", "decode_window", "decode_shared", "make_shared_workspace",
    "pages_workspace_size", "make_pages_workspace", "pages_copy", "pages_fork", "pages_alloc",
    "pages_free", "pages_compact", "PAGES_BAD_ENTRY", "PAGES_FULL",
    "kv_append_chunk", "kv_read", "prefill_chunk", "prefill_expanded", "make_prefill_workspace",
]

LSE_NATURAL = 0
LSE_BASE2 = 1
KV_BF16 = 0
KV_E4M3 = 1
PAGES_BAD_ENTRY = 1
PAGES_FULL = 2
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_lib", "libmla_decode.so")
_lib = None
_lock = threading.Lock()


class MlaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


class DecodeDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("q_len", ctypes.c_int32), ("head_dim_qk", ctypes.c_int32),
                ("head_dim_v", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("kv_scale", ctypes.c_float)]


class CombineDesc(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("lse_base", ctypes.c_int32),
                ("out_lse", ctypes.c_void_p)]


def library_path() -> str:
    return _LIB_PATH


class DcpMetaDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_req_slots", ctypes.c_int32),
                ("req_to_token_width", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("extra_tokens", ctypes.c_int32), ("pad_value", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class PagesDesc(ctypes.Structure):
    _fields_ = [("num_requests", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim_qk", ctypes.c_int32), ("kv_dtype", ctypes.c_int32)]


class ExpandedDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("q_tokens", ctypes.c_int32),
                ("k_tokens", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("rope_token_stride", ctypes.c_int64), ("v_token_stride", ctypes.c_int64),
                ("v_head_stride", ctypes.c_int64)]


def load_library():
    """Loads the built library (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is not built; run `python -m mla_paged_decode_gb300.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.mla_decode_partial.argtypes = [vp, vp, vp, vp, i32, i32, f32, i32, vp, vp,
                                           ctypes.POINTER(DecodeDesc), vp, sz, vp]
        lib.mla_decode_partial.restype = i32
        lib.mla_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeDesc), i32]
        lib.mla_decode_workspace_size.restype = sz
        lib.mla_decode_check_workspace.argtypes = [vp, vp]
        lib.mla_decode_check_workspace.restype = i32
        lib.mla_decode_dcp.argtypes = [vp, vp, vp, vp, i32, f32, i32, vp, vp, vp, vp,
                                       ctypes.POINTER(DecodeDesc), vp, sz, vp]
        lib.mla_decode_dcp.restype = i32
        lib.mla_decode_dcp_workspace_size.argtypes = [ctypes.POINTER(DecodeDesc), i32, i32]
        lib.mla_decode_dcp_workspace_size.restype = sz
        lib.mla_dcp_local_metadata.argtypes = [vp, vp, vp, i32, i32, ctypes.POINTER(DcpMetaDesc),
                                               vp, vp, vp, vp, vp]
        lib.mla_dcp_local_metadata.restype = i32
        lib.mla_kv_append.argtypes = [vp, vp, vp, vp, i32, i32, ctypes.POINTER(DecodeDesc), vp, vp]
        lib.mla_kv_append.restype = i32
        lib.mla_lse_combine.argtypes = [vp, vp, i32, vp, ctypes.POINTER(CombineDesc), vp]
        lib.mla_lse_combine.restype = i32
        dd = ctypes.POINTER(DecodeDesc)
        lib.mla_decode_window.argtypes = [vp, vp, vp, vp, i32, i32, f32, i32, vp, vp, dd, vp, sz, vp]
        lib.mla_decode_window.restype = i32
        lib.mla_decode_shared_workspace_size.argtypes = [dd, i32, i32]
        lib.mla_decode_shared_workspace_size.restype = sz
        lib.mla_decode_shared.argtypes = [vp, vp, vp, vp, vp, vp, i32, f32, i32, vp, vp, dd, vp, sz, vp]
        lib.mla_decode_shared.restype = i32
        pd = ctypes.POINTER(PagesDesc)
        lib.mla_pages_workspace_size.argtypes = [i32]
        lib.mla_pages_workspace_size.restype = sz
        lib.mla_pages_copy.argtypes = [vp, vp, vp, vp, i32, i32, pd, vp, vp]
        lib.mla_pages_fork.argtypes = [vp, vp, vp, vp, vp, vp, i32, pd, vp, sz, vp, vp]
        lib.mla_pages_alloc.argtypes = [vp, vp, vp, vp, pd, vp, sz, vp, vp]
        lib.mla_pages_free.argtypes = [vp, vp, vp, vp, i32, i32, pd, vp, vp]
        lib.mla_pages_compact.argtypes = [vp, vp, vp, vp, pd, vp, sz, vp, vp]
        for f in (lib.mla_pages_copy, lib.mla_pages_fork, lib.mla_pages_alloc, lib.mla_pages_free,
                  lib.mla_pages_compact):
            f.restype = i32
        i64 = ctypes.c_int64
        lib.mla_kv_append_chunk.argtypes = [vp, i64, i32, vp, vp, vp, vp, i32, i32, dd, vp, vp]
        lib.mla_kv_append_chunk.restype = i32
        lib.mla_kv_read.argtypes = [vp, vp, vp, vp, vp, i64, i32, dd, vp, vp]
        lib.mla_kv_read.restype = i32
        lib.mla_prefill_workspace_size.argtypes = [i32]
        lib.mla_prefill_workspace_size.restype = sz
        lib.mla_prefill_chunk.argtypes = [vp, i32, vp, vp, vp, vp, f32, i32, vp, vp, dd, vp, sz, vp]
        lib.mla_prefill_chunk.restype = i32
        lib.mla_prefill_expanded.argtypes = [vp, vp, vp, vp, vp, vp, f32, i32, vp, vp, ctypes.POINTER(ExpandedDesc),
                                             vp, sz, vp]
        lib.mla_prefill_expanded.restype = i32
        lib.mla_status_string.argtypes = [i32]
        lib.mla_status_string.restype = ctypes.c_char_p
        lib.mla_last_cuda_error.argtypes = []
        lib.mla_last_cuda_error.restype = ctypes.c_char_p
        lib.mla_version.argtypes = []
        lib.mla_version.restype = i32
        lib.mla_selftest_bounded_wait.argtypes = [vp, ctypes.c_int64, vp]
        lib.mla_selftest_bounded_wait.restype = i32
        _lib = lib
        return lib


def _check(status: int):
    if status != 0:
        lib = load_library()
        msg = lib.mla_status_string(status).decode()
        if status == -7:
            msg += ": " + lib.mla_last_cuda_error().decode()
        raise MlaError(status, msg)


def _int32(value, name: str) -> int:
    """An integer argument of the C calls; ctypes would cut a larger one to its
    low 32 bits without a word (a window of 2**32 + 7 tokens to 7)."""
    v = int(value)
    if not -0x80000000 <= v <= 0x7fffffff:
        raise ValueError(f"{name} = {v} does not fit into 32 bits")
    return v


# The current stream's handle and the current device without the Python
# objects around them (2 us and 0.4 us of a small call's host time).
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda index: torch.cuda.current_stream(index).cuda_stream
_NO_SWITCH = contextlib.nullcontext()


def _on(device):
    """The device context for a call: nothing to switch when it is current
    (the switch costs a few microseconds, felt by small decodes)."""
    if torch.cuda.current_device() == device.index:
        return _NO_SWITCH
    return torch.cuda.device(device)


def _stream_ptr(stream, device) -> int:
    return int(stream.cuda_stream) if stream is not None else _raw_stream(device.index)


def _allocating_on(stream, device):
    """The context in which a call that runs on `stream` allocates what it was
    not given.  The caching allocator orders a block by the stream it was
    allocated on: scratch from the current stream's pool, dropped when the call
    returns, could go to that stream's next tensor while the kernels on
    `stream` still use it, and its zero fill could run after them."""
    if stream is None or int(stream.cuda_stream) == _raw_stream(device.index):
        return _NO_SWITCH
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream), device=device)
    return torch.cuda.stream(stream)


def _output(shape, dtype, device, stream):
    """An output that the caller did not give: allocated on the call's stream
    and kept, when it is dropped, until the current stream is done with it."""
    where = _allocating_on(stream, device)
    if where is _NO_SWITCH:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with where:
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _launch(fn, device, stream, *args):
    """fn(*args, stream) on the tensors' device; raises on a bad status."""
    s = _stream_ptr(stream, device)
    if torch.cuda.current_device() == device.index:
        st = fn(*args, s)
    else:
        with torch.cuda.device(device):
            st = fn(*args, s)
    if st != 0:
        _check(st)


def _kv_dtype_code(kv_pages: torch.Tensor) -> int:
    if kv_pages.dtype == torch.bfloat16:
        return KV_BF16
    if kv_pages.dtype in (torch.uint8, torch.float8_e4m3fn):
        return KV_E4M3
    raise TypeError(f"kv_pages must be bf16 or e4m3 bytes, got {kv_pages.dtype}")


_KV_TYPES = (torch.bfloat16, torch.uint8, torch.float8_e4m3fn)
_I32 = (torch.int32,)
_DESCS: dict = {}


def _decode_desc(q, kv_pages, block_table, kv_scale) -> DecodeDesc:
    """The call's size descriptor, built once per distinct set of shapes (the
    library only reads it during the call)."""
    key = (q.shape, kv_pages.shape, kv_pages.dtype, block_table.shape, float(kv_scale))
    d = _DESCS.get(key)
    if d is None:
        d = _make_decode_desc(q, kv_pages, block_table, kv_scale)
        if len(_DESCS) > 256:
            _DESCS.clear()
        _DESCS[key] = d
    return d


def _make_decode_desc(q, kv_pages, block_table, kv_scale) -> DecodeDesc:
    if q.dim() != 4:
        raise ValueError("q must be [B, q_len, H, 576]")
    B, q_len, H, dqk = (_int32(n, "a size of q") for n in q.shape)
    if kv_pages.dim() != 3:
        raise ValueError("kv_pages must be [num_pages, page_size, 576]")
    return DecodeDesc(batch=B, num_heads=H, q_len=q_len, head_dim_qk=dqk, head_dim_v=512,
                      page_size=_int32(kv_pages.shape[1], "page_size"),
                      num_pages=_int32(kv_pages.shape[0], "num_pages"),
                      max_pages_per_seq=_int32(block_table.shape[1], "max_pages") if block_table.dim() == 2 else 0,
                      kv_dtype=_kv_dtype_code(kv_pages), kv_scale=float(kv_scale))


def workspace_size(q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                   kv_scale: float = 1.0) -> int:
    d = _decode_desc(q, kv_pages, block_table, kv_scale)
    with torch.cuda.device(q.device):
        n = load_library().mla_decode_workspace_size(ctypes.byref(d), 0)
    if n == 0:
        raise MlaError(-2, "cannot size a workspace for these shapes")
    return n


def make_workspace(q, kv_pages, block_table, kv_scale: float = 1.0) -> torch.Tensor:
    """A zero-filled workspace for these shapes on q's device."""
    return torch.zeros(workspace_size(q, kv_pages, block_table, kv_scale), dtype=torch.uint8,
                       device=q.device)


def _need(t: torch.Tensor, name: str, dtypes, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def decode_partial(q, kv_pages, block_table, seq_lens, part_id: int, num_parts: int,
                   sm_scale: float, lse_base: int, out, lse, *, kv_scale: float = 1.0,
                   workspace: torch.Tensor | None = None, stream=None):
    """mla_decode_partial on torch tensors (see include/mla_decode.h).

    q bf16 [B,1,H,576]; kv_pages bf16 [pages,64,576] or uint8/float8_e4m3fn;
    block_table int32 [B,max_pages]; seq_lens int32 [B] (global lengths);
    out bf16 [B,1,H,512] and lse fp32 [B,1,H] are written in place.
    """
    part_id, num_parts = _int32(part_id, "part_id"), _int32(num_parts, "num_parts")
    lse_base = _int32(lse_base, "lse_base")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("decode_partial runs on CUDA tensors only")
    _need(q, "q", (torch.bfloat16,), dev)
    _need(kv_pages, "kv_pages", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn), dev)
    _need(block_table, "block_table", (torch.int32,), dev)
    _need(seq_lens, "seq_lens", (torch.int32,), dev)
    _need(out, "out", (torch.bfloat16,), dev)
    _need(lse, "lse", (torch.float32,), dev)
    d = _decode_desc(q, kv_pages, block_table, kv_scale)
    if seq_lens.numel() != d.batch or block_table.dim() != 2 or block_table.shape[0] != d.batch:
        raise ValueError("seq_lens / block_table do not match the batch")
    if out.numel() != d.batch * d.q_len * d.num_heads * 512 or lse.numel() != d.batch * d.q_len * d.num_heads:
        raise ValueError("out must be [B,1,H,512] and lse [B,1,H]")
    if workspace is None:
        with _allocating_on(stream, dev):
            workspace = make_workspace(q, kv_pages, block_table, kv_scale)
    _need(workspace, "workspace", (torch.uint8,), dev)
    with _on(dev):
        st = load_library().mla_decode_partial(
            q.data_ptr(), kv_pages.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
            part_id, num_parts, float(sm_scale), lse_base, out.data_ptr(),
            lse.data_ptr(), ctypes.byref(d), workspace.data_ptr(), workspace.numel(),
            _stream_ptr(stream, dev))
    _check(st)
    return out, lse


def kv_append(kv_new, kv_pages, block_table, positions, part_id: int = 0, num_parts: int = 1, *,
              kv_scale: float = 1.0, error_word=None, stream=None):
    """mla_kv_append on torch tensors (see include/mla_decode.h).

    kv_new bf16 [B, 576] (or [B, 1, 576]): each request's new token row;
    positions int32 [B]: its global index (the length before the append;
    negative skips the request).  Row positions[b] is written into kv_pages
    (bf16, or uint8/float8_e4m3fn quantised with kv_scale) in place, if
    partition part_id of num_parts owns it.  error_word: optional int32 [1]
    device tensor that receives bit 0 for a row whose page entry is out of
    range (that row is skipped).
    """
    part_id, num_parts = _int32(part_id, "part_id"), _int32(num_parts, "num_parts")
    dev = kv_pages.device
    if dev.type != "cuda":
        raise ValueError("kv_append runs on CUDA tensors only")
    _need(kv_new, "kv_new", (torch.bfloat16,), dev)
    _need(kv_pages, "kv_pages", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn), dev)
    _need(block_table, "block_table", (torch.int32,), dev)
    _need(positions, "positions", (torch.int32,), dev)
    if kv_pages.dim() != 3 or block_table.dim() != 2:
        raise ValueError("kv_pages must be [num_pages, 64, 576] and block_table [B, max_pages]")
    B = positions.numel()
    if kv_new.numel() != B * 576 or kv_new.shape[-1] != 576 or block_table.shape[0] != B:
        raise ValueError("kv_new must be [B, 576] and block_table [B, max_pages] for B positions")
    if error_word is not None:
        _need(error_word, "error_word", (torch.int32,), dev)
    d = DecodeDesc(batch=_int32(B, "batch"), num_heads=1, q_len=1, head_dim_qk=576, head_dim_v=512,
                   page_size=_int32(kv_pages.shape[1], "page_size"), num_pages=_int32(kv_pages.shape[0], "num_pages"),
                   max_pages_per_seq=_int32(block_table.shape[1], "max_pages"), kv_dtype=_kv_dtype_code(kv_pages),
                   kv_scale=float(kv_scale))
    with _on(dev):
        st = load_library().mla_kv_append(
            kv_new.data_ptr(), kv_pages.data_ptr(), block_table.data_ptr(), positions.data_ptr(),
            part_id, num_parts, ctypes.byref(d),
            error_word.data_ptr() if error_word is not None else None, _stream_ptr(stream, dev))
    _check(st)
    return kv_pages


def make_dcp_workspace(q, kv_pages, block_table, num_parts: int, kv_scale: float = 1.0):
    """A zero-filled workspace for decode_dcp over num_parts partitions."""
    d = _decode_desc(q, kv_pages, block_table, kv_scale)
    with torch.cuda.device(q.device):
        n = load_library().mla_decode_dcp_workspace_size(ctypes.byref(d), _int32(num_parts, "num_parts"), 0)
    if n == 0:
        raise MlaError(-2, "cannot size a workspace for these shapes")
    return torch.zeros(n, dtype=torch.uint8, device=q.device)


def decode_dcp(q, kv_pages, block_table, seq_lens, num_parts: int, sm_scale: float,
               lse_base: int, *, partials=None, partial_lses=None, out=None, out_lse=None,
               kv_scale: float = 1.0, workspace=None, stream=None):
    """mla_decode_dcp: every partition's (out, lse) and their merge in one call.

    Returns (out [B,1,H,512], out_lse [B,1,H] or None, partials [P,B,1,H,512],
    partial_lses [P,B,1,H]); the output tensors are allocated when not given.
    """
    num_parts, lse_base = _int32(num_parts, "num_parts"), _int32(lse_base, "lse_base")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("decode_dcp runs on CUDA tensors only")
    _need(q, "q", (torch.bfloat16,), dev)
    _need(kv_pages, "kv_pages", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn), dev)
    _need(block_table, "block_table", (torch.int32,), dev)
    _need(seq_lens, "seq_lens", (torch.int32,), dev)
    d = _decode_desc(q, kv_pages, block_table, kv_scale)
    B, T, H, P = d.batch, d.q_len, d.num_heads, num_parts
    if seq_lens.numel() != B or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("seq_lens / block_table do not match the batch")
    if partials is None:
        partials = _output((P, B, T, H, 512), torch.bfloat16, dev, stream)
    if partial_lses is None:
        partial_lses = _output((P, B, T, H), torch.float32, dev, stream)
    if out is None:
        out = _output((B, T, H, 512), torch.bfloat16, dev, stream)
    _need(partials, "partials", (torch.bfloat16,), dev)
    _need(partial_lses, "partial_lses", (torch.float32,), dev)
    _need(out, "out", (torch.bfloat16,), dev)
    if partials.numel() != P * B * T * H * 512 or partial_lses.numel() != P * B * T * H:
        raise ValueError("partials must be [P,B,q_len,H,512] and partial_lses [P,B,q_len,H]")
    if out.numel() != B * T * H * 512:
        raise ValueError("out must be [B,q_len,H,512]")
    if out_lse is not None:
        _need(out_lse, "out_lse", (torch.float32,), dev)
        if out_lse.numel() != B * T * H:
            raise ValueError("out_lse must be [B,q_len,H]")
    if workspace is None:
        with _allocating_on(stream, dev):
            workspace = make_dcp_workspace(q, kv_pages, block_table, P, kv_scale)
    _need(workspace, "workspace", (torch.uint8,), dev)
    with _on(dev):
        st = load_library().mla_decode_dcp(
            q.data_ptr(), kv_pages.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), P,
            float(sm_scale), lse_base, partials.data_ptr(), partial_lses.data_ptr(),
            out.data_ptr(), out_lse.data_ptr() if out_lse is not None else None, ctypes.byref(d),
            workspace.data_ptr(), workspace.numel(), _stream_ptr(stream, dev))
    _check(st)
    return out, out_lse, partials, partial_lses


def dcp_local_metadata(seq_lens, req_pool_indices, req_to_token, part_id: int, num_parts: int,
                       *, max_pages: int, extra_tokens: int = 0, pad_value: int = 0,
                       global_lens=None, local_lens=None, block_table=None, error_word=None,
                       stream=None):
    """mla_dcp_local_metadata: a DCP rank's global and local lengths and its
    rank-local page table [B, max_pages], built on the device (into the given
    buffers when passed, so a captured graph can keep reading them).
    Returns (global_lens, local_lens, block_table)."""
    part_id, num_parts = _int32(part_id, "part_id"), _int32(num_parts, "num_parts")
    max_pages, extra_tokens = _int32(max_pages, "max_pages"), _int32(extra_tokens, "extra_tokens")
    pad_value = _int32(pad_value, "pad_value")
    dev = seq_lens.device
    if dev.type != "cuda":
        raise ValueError("dcp_local_metadata runs on CUDA tensors only")
    _need(seq_lens, "seq_lens", (torch.int32,), dev)
    _need(req_pool_indices, "req_pool_indices", (torch.int32,), dev)
    _need(req_to_token, "req_to_token", (torch.int32,), dev)
    B = seq_lens.numel()
    if req_pool_indices.numel() != B or req_to_token.dim() != 2:
        raise ValueError("req_pool_indices must be [B] and req_to_token [slots, width]")
    global_lens = global_lens if global_lens is not None else _output((B,), torch.int32, dev, stream)
    local_lens = local_lens if local_lens is not None else _output((B,), torch.int32, dev, stream)
    block_table = block_table if block_table is not None else _output((B, max_pages), torch.int32, dev, stream)
    for t, n in ((global_lens, "global_lens"), (local_lens, "local_lens"), (block_table, "block_table")):
        _need(t, n, (torch.int32,), dev)
    if global_lens.numel() != B or local_lens.numel() != B or block_table.numel() != B * max_pages:
        raise ValueError("output buffers do not match the batch and max_pages")
    if error_word is not None:
        _need(error_word, "error_word", (torch.int32,), dev)
    d = DcpMetaDesc(batch=_int32(B, "batch"), num_req_slots=_int32(req_to_token.shape[0], "slots"),
                    req_to_token_width=_int32(req_to_token.shape[1], "width"), max_pages_per_seq=max_pages,
                    extra_tokens=extra_tokens, pad_value=pad_value, page_size=64)
    with _on(dev):
        st = load_library().mla_dcp_local_metadata(
            seq_lens.data_ptr(), req_pool_indices.data_ptr(), req_to_token.data_ptr(), part_id,
            num_parts, ctypes.byref(d), global_lens.data_ptr(), local_lens.data_ptr(),
            block_table.data_ptr(), error_word.data_ptr() if error_word is not None else None,
            _stream_ptr(stream, dev))
    _check(st)
    return global_lens, local_lens, block_table


def check_workspace(workspace: torch.Tensor, stream=None) -> int:
    """Synchronises the stream and returns (and clears) the kernel's bounds
    status: 0, or -9 if a block-table entry or a length was out of bounds."""
    with torch.cuda.device(workspace.device):
        st = load_library().mla_decode_check_workspace(workspace.data_ptr(),
                                                       _stream_ptr(stream, workspace.device))
    if st not in (0, -9):
        _check(st)
    return st


def selftest_bounded_wait(workspace: torch.Tensor, timeout_ns: int, stream=None) -> None:
    """mla_selftest_bounded_wait: two warps wait on barriers that nothing
    completes; the waits give up (after timeout_ns, and on the abort flag)
    and report MLA_ERR_TIMEOUT in the workspace's error word."""
    with torch.cuda.device(workspace.device):
        _check(load_library().mla_selftest_bounded_wait(
            workspace.data_ptr(), int(timeout_ns), _stream_ptr(stream, workspace.device)))


def lse_combine(partials, lses, num_parts: int, out, *, lse_base: int = LSE_NATURAL,
                out_lse=None, stream=None):
    """mla_lse_combine: partials bf16 [P,T,H,D], lses fp32 [P,T,H] -> out bf16 [T,H,D]."""
    num_parts, lse_base = _int32(num_parts, "num_parts"), _int32(lse_base, "lse_base")
    dev = partials.device
    if dev.type != "cuda":
        raise ValueError("lse_combine runs on CUDA tensors only")
    _need(partials, "partials", (torch.bfloat16,), dev)
    _need(lses, "lses", (torch.float32,), dev)
    _need(out, "out", (torch.bfloat16,), dev)
    if partials.dim() != 4 or partials.shape[0] != num_parts:
        raise ValueError("partials must be [num_parts, T, H, D]")
    P, T, H, D = partials.shape
    if lses.numel() != P * T * H or out.numel() != T * H * D:
        raise ValueError("lses must be [P,T,H] and out [T,H,D]")
    if out_lse is not None:
        _need(out_lse, "out_lse", (torch.float32,), dev)
        if out_lse.numel() != T * H:
            raise ValueError("out_lse must be [T,H]")
    d = CombineDesc(num_tokens=_int32(T, "tokens"), num_heads=_int32(H, "heads"), head_dim=_int32(D, "head_dim"),
                    lse_base=lse_base,
                    out_lse=out_lse.data_ptr() if out_lse is not None else None)
    with _on(dev):
        st = load_library().mla_lse_combine(partials.data_ptr(), lses.data_ptr(), num_parts,
                                            out.data_ptr(), ctypes.byref(d), _stream_ptr(stream, dev))
    _check(st)
    return out


def decode_partial_noalloc(q, kv_pages, block_table, seq_lens, part_id: int, num_parts: int,
                           sm_scale: float, lse_base: int, out, lse, *, kv_scale: float = 1.0,
                           stream=None):
    """mla_decode_partial_noalloc: the same call without a workspace, for
    callers that cannot allocate device memory (see include/mla_decode.h).
    It uses scratch built into the library, shared by every call: calls that
    may overlap on the GPU must be serialised by the caller."""
    part_id, num_parts = _int32(part_id, "part_id"), _int32(num_parts, "num_parts")
    lse_base = _int32(lse_base, "lse_base")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("decode_partial_noalloc runs on CUDA tensors only")
    _need(q, "q", (torch.bfloat16,), dev)
    _need(kv_pages, "kv_pages", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn), dev)
    _need(block_table, "block_table", (torch.int32,), dev)
    _need(seq_lens, "seq_lens", (torch.int32,), dev)
    _need(out, "out", (torch.bfloat16,), dev)
    _need(lse, "lse", (torch.float32,), dev)
    d = _decode_desc(q, kv_pages, block_table, kv_scale)
    lib = load_library()
    fn = lib.mla_decode_partial_noalloc
    vp, i32 = ctypes.c_void_p, ctypes.c_int
    fn.argtypes = [vp, vp, vp, vp, i32, i32, ctypes.c_float, i32, vp, vp,
                   ctypes.POINTER(DecodeDesc), vp]
    fn.restype = i32
    with _on(dev):
        st = fn(q.data_ptr(), kv_pages.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                part_id, num_parts, float(sm_scale), lse_base, out.data_ptr(),
                lse.data_ptr(), ctypes.byref(d), _stream_ptr(stream, dev))
    _check(st)
    return out, lse


def _view_args(what, q, kv_pages, block_table, seq_lens, out, lse, kv_scale):
    """Checks what decode_window and decode_shared have in common; returns the
    device and the descriptor."""
    dev = q.device
    if dev.type != "cuda":
        raise ValueError(f"{what} runs on CUDA tensors only")
    _need(q, "q", (torch.bfloat16,), dev)
    _need(kv_pages, "kv_pages", _KV_TYPES, dev)
    _need(block_table, "block_table", (torch.int32,), dev)
    _need(seq_lens, "seq_lens", (torch.int32,), dev)
    _need(out, "out", (torch.bfloat16,), dev)
    _need(lse, "lse", (torch.float32,), dev)
    d = _decode_desc(q, kv_pages, block_table, kv_scale)
    if seq_lens.numel() != d.batch or block_table.dim() != 2 or block_table.shape[0] != d.batch:
        raise ValueError("seq_lens / block_table do not match the batch")
    if kv_pages.shape[2] != 576:
        raise ValueError("kv_pages must be [num_pages, 64, 576]")
    rows = d.batch * d.q_len * d.num_heads
    if out.numel() != rows * 512 or lse.numel() != rows:
        raise ValueError("out must be [B,q_len,H,512] and lse [B,q_len,H]")
    return dev, d


def decode_window(q, kv_pages, block_table, seq_lens, window: int, sinks: int, sm_scale: float,
                  lse_base: int, out, lse, *, kv_scale: float = 1.0, workspace=None, stream=None):
    """mla_decode_window: each query sees the last `window` tokens up to its
    own and the request's first `sinks` tokens.  Tensors as for
    decode_partial (q [B,q_len,H,576], 1..16 query tokens); the workspace is
    make_workspace's.  Entries of pages out of view may be -1."""
    window, sinks, lse_base = _int32(window, "window"), _int32(sinks, "sinks"), _int32(lse_base, "lse_base")
    dev, d = _view_args("decode_window", q, kv_pages, block_table, seq_lens, out, lse, kv_scale)
    if workspace is None:
        with _allocating_on(stream, dev):
            workspace = make_workspace(q, kv_pages, block_table, kv_scale)
    _need(workspace, "workspace", (torch.uint8,), dev)
    _launch(load_library().mla_decode_window, dev, stream, q.data_ptr(), kv_pages.data_ptr(),
            block_table.data_ptr(), seq_lens.data_ptr(), window, sinks, float(sm_scale),
            lse_base, out.data_ptr(), lse.data_ptr(), ctypes.byref(d), workspace.data_ptr(),
            workspace.numel())
    return out, lse


def make_shared_workspace(q, kv_pages, block_table, num_groups: int, kv_scale: float = 1.0):
    """A zero-filled workspace for decode_shared over num_groups groups."""
    d = _decode_desc(q, kv_pages, block_table, kv_scale)
    with torch.cuda.device(q.device):
        n = load_library().mla_decode_shared_workspace_size(ctypes.byref(d), _int32(num_groups, "num_groups"), 0)
    if n == 0:
        raise MlaError(-2, "cannot size a workspace for these shapes")
    return torch.zeros(n, dtype=torch.uint8, device=q.device)


def decode_shared(q, kv_pages, block_table, seq_lens, group_starts, shared_pages, sm_scale: float,
                  lse_base: int, out, lse, *, kv_scale: float = 1.0, workspace=None, stream=None):
    """mla_decode_shared: the requests group_starts[g] .. group_starts[g + 1]
    (int32 [G + 1], from 0 to B) have their first shared_pages[g] (int32 [G])
    pages in common, which are read and multiplied once for the group.
    Tensors as for decode_partial; the workspace is make_shared_workspace's."""
    lse_base = _int32(lse_base, "lse_base")
    dev, d = _view_args("decode_shared", q, kv_pages, block_table, seq_lens, out, lse, kv_scale)
    _need(group_starts, "group_starts", (torch.int32,), dev)
    _need(shared_pages, "shared_pages", (torch.int32,), dev)
    groups = shared_pages.numel()
    if groups < 1 or group_starts.numel() != groups + 1:
        raise ValueError("group_starts must be [G + 1] and shared_pages [G], G >= 1")
    if workspace is None:
        with _allocating_on(stream, dev):
            workspace = make_shared_workspace(q, kv_pages, block_table, groups, kv_scale)
    _need(workspace, "workspace", (torch.uint8,), dev)
    _launch(load_library().mla_decode_shared, dev, stream, q.data_ptr(), kv_pages.data_ptr(),
            block_table.data_ptr(), seq_lens.data_ptr(), group_starts.data_ptr(), shared_pages.data_ptr(),
            _int32(groups, "groups"), float(sm_scale), lse_base, out.data_ptr(), lse.data_ptr(), ctypes.byref(d),
            workspace.data_ptr(), workspace.numel())
    return out, lse


_CACHE_DESCS: dict = {}


def _cache_desc(batch, heads, kv_pages, block_table, kv_scale):
    """The size descriptor (by reference) of a call whose queries are not
    [B, q_len, H, 576], built once per set of sizes."""
    key = (batch, heads, kv_pages.shape, kv_pages.dtype, block_table.shape, float(kv_scale))
    d = _CACHE_DESCS.get(key)
    if d is None:
        if kv_pages.dim() != 3 or kv_pages.shape[2] != 576:
            raise ValueError("kv_pages must be [num_pages, 64, 576]")
        if block_table.dim() != 2 or block_table.shape[0] != batch:
            raise ValueError("block_table must be [B, max_pages]")
        if len(_CACHE_DESCS) > 256:
            _CACHE_DESCS.clear()
        d = _CACHE_DESCS[key] = DecodeDesc(
            batch=_int32(batch, "batch"), num_heads=_int32(heads, "heads"), q_len=1, head_dim_qk=576, head_dim_v=512,
            page_size=_int32(kv_pages.shape[1], "page_size"), num_pages=_int32(kv_pages.shape[0], "num_pages"),
            max_pages_per_seq=_int32(block_table.shape[1], "max_pages"), kv_dtype=_kv_dtype_code(kv_pages),
            kv_scale=float(kv_scale))
    return ctypes.byref(d)


def _chunk_args(what, rows, rows_name, kv_pages, block_table, starts, starts_name, positions, kv_scale, error_word):
    """Checks what kv_append_chunk and kv_read have in common; returns the
    device, the descriptor, the row stride and the number of rows."""
    dev = kv_pages.device
    if dev.type != "cuda":
        raise ValueError(f"{what} runs on CUDA tensors only")
    _need(kv_pages, "kv_pages", _KV_TYPES, dev)
    _ints(block_table, "block_table", dev, 2)
    _ints(starts, starts_name, dev, 1)
    _ints(positions, "positions", dev, 1)
    if not isinstance(rows, torch.Tensor) or rows.dtype != torch.bfloat16:
        raise TypeError(f"{rows_name} must be a bf16 tensor")
    if rows.device != dev:
        raise ValueError(f"{rows_name} is on {rows.device}, expected {dev}")
    if rows.dim() != 2 or rows.shape[1] != 576 or rows.stride(1) != 1:
        raise ValueError(f"{rows_name} must be [N, 576] with rows of consecutive values")
    B, n = positions.numel(), rows.shape[0]
    if starts.numel() != B + 1:
        raise ValueError(f"{starts_name} must be [B + 1] for B positions")
    if error_word is not None:
        _need(error_word, "error_word", _I32, dev)
    return dev, _cache_desc(B, 1, kv_pages, block_table, kv_scale), rows.stride(0) if n > 1 else 576, \
        _int32(n, "rows")


def kv_append_chunk(kv_new, kv_pages, block_table, chunk_starts, positions, part_id: int = 0, num_parts: int = 1,
                    *, kv_scale: float = 1.0, error_word=None, stream=None):
    """mla_kv_append_chunk: rows chunk_starts[b] .. chunk_starts[b + 1] (int32
    [B + 1]) of kv_new bf16 [N, 576] become request b's tokens positions[b]
    (int32 [B]; negative skips the request), positions[b] + 1, ... in kv_pages
    (bf16, or e4m3 quantised with kv_scale), where partition part_id of
    num_parts owns them.  Rows of kv_new may lie inside wider ones.  Into
    error_word (int32 [1]) goes bit 0 for rows without a page and bit 1 for
    starts that fall or leave kv_new."""
    part_id, num_parts = _int32(part_id, "part_id"), _int32(num_parts, "num_parts")
    dev, d, stride, n = _chunk_args("kv_append_chunk", kv_new, "kv_new", kv_pages, block_table, chunk_starts,
                                    "chunk_starts", positions, kv_scale, error_word)
    _launch(load_library().mla_kv_append_chunk, dev, stream, kv_new.data_ptr(), stride, n, kv_pages.data_ptr(),
            block_table.data_ptr(), chunk_starts.data_ptr(), positions.data_ptr(), part_id, num_parts, d,
            _opt(error_word))
    return kv_pages


def kv_read(kv_pages, block_table, read_starts, positions, out, *, kv_scale: float = 1.0, error_word=None,
            stream=None):
    """mla_kv_read: request b's cached tokens positions[b] (int32 [B]), ... go
    to rows read_starts[b] .. read_starts[b + 1] (int32 [B + 1]) of out bf16
    [N, 576], e4m3 codes times kv_scale.  Other rows of out stay as they are.
    error_word as for kv_append_chunk; rows without a page become zeros.  The
    rows of all partitions are read: the pool has to hold them."""
    dev, d, stride, n = _chunk_args("kv_read", out, "out", kv_pages, block_table, read_starts, "read_starts",
                                    positions, kv_scale, error_word)
    _launch(load_library().mla_kv_read, dev, stream, kv_pages.data_ptr(), block_table.data_ptr(),
            read_starts.data_ptr(), positions.data_ptr(), out.data_ptr(), stride, n, d, _opt(error_word))
    return out


def make_prefill_workspace(q) -> torch.Tensor:
    """A zero-filled workspace for prefill_chunk and prefill_expanded on q's
    device; its size does not depend on the batch."""
    with torch.cuda.device(q.device):
        n = load_library().mla_prefill_workspace_size(0)
    if n == 0:
        raise MlaError(-8, "cannot size a workspace on this device")
    return torch.zeros(n, dtype=torch.uint8, device=q.device)


def _prefill_outputs(out, lse, dev, tokens, heads, dim, workspace, stream, q):
    _need(out, "out", (torch.bfloat16,), dev)
    _need(lse, "lse", (torch.float32,), dev)
    if out.shape != (tokens, heads, dim) or lse.shape != (tokens, heads):
        raise ValueError(f"out must be [N, H, {dim}] and lse [N, H]")
    if workspace is None:
        with _allocating_on(stream, dev):
            workspace = make_prefill_workspace(q)
    _need(workspace, "workspace", (torch.uint8,), dev)
    return workspace


def prefill_chunk(q, kv_pages, block_table, seq_lens, chunk_starts, sm_scale: float, lse_base: int, out, lse, *,
                  kv_scale: float = 1.0, workspace=None, stream=None):
    """mla_prefill_chunk: tokens chunk_starts[b] .. chunk_starts[b + 1] (int32
    [B + 1]) of q bf16 [N, H, 576] are the last of request b's seq_lens[b]
    cached tokens and attend to those up to themselves; out bf16 [N, H, 512]
    and lse fp32 [N, H] are written in place, tokens of no request left as
    they are.  The pool has to hold the rows of all partitions.  The workspace
    is make_prefill_workspace's."""
    lse_base = _int32(lse_base, "lse_base")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("prefill_chunk runs on CUDA tensors only")
    _need(q, "q", (torch.bfloat16,), dev)
    _need(kv_pages, "kv_pages", _KV_TYPES, dev)
    _ints(block_table, "block_table", dev, 2)
    _ints(seq_lens, "seq_lens", dev, 1)
    _ints(chunk_starts, "chunk_starts", dev, 1)
    if q.dim() != 3 or q.shape[2] != 576:
        raise ValueError("q must be [N, H, 576]")
    n, heads, _ = q.shape
    B = seq_lens.numel()
    if chunk_starts.numel() != B + 1:
        raise ValueError("chunk_starts must be [B + 1] for B lengths")
    d = _cache_desc(B, heads, kv_pages, block_table, kv_scale)
    workspace = _prefill_outputs(out, lse, dev, n, heads, 512, workspace, stream, q)
    _launch(load_library().mla_prefill_chunk, dev, stream, q.data_ptr(), _int32(n, "tokens"), kv_pages.data_ptr(),
            block_table.data_ptr(), seq_lens.data_ptr(), chunk_starts.data_ptr(), float(sm_scale), lse_base,
            out.data_ptr(), lse.data_ptr(), d, workspace.data_ptr(), workspace.numel())
    return out, lse


_EXPANDED_DESCS: dict = {}


def _stride(t, dim, least):
    """A stride for the library: that of a dimension of one index may be
    anything and is not used."""
    return t.stride(dim) if t.shape[dim] > 1 else least


def _expanded_desc(q, k_nope, k_rope, v, batch, causal):
    """Checks the four tensors, once per set of layouts, and returns the
    call's descriptor (by reference)."""
    if not all(isinstance(t, torch.Tensor) for t in (q, k_nope, k_rope, v)):
        raise TypeError("q, k_nope, k_rope and v must be tensors")
    key = (q.shape, q.stride(), q.dtype, q.device, k_nope.shape, k_nope.stride(), k_nope.dtype, k_nope.device,
           k_rope.shape, k_rope.stride(), k_rope.dtype, k_rope.device, v.shape, v.stride(), v.dtype, v.device,
           batch, causal)
    d = _EXPANDED_DESCS.get(key)
    if d is None:
        for t, name in ((q, "q"), (k_nope, "k_nope"), (k_rope, "k_rope"), (v, "v")):
            if t.dtype != torch.bfloat16:
                raise TypeError(f"{name} must be a bf16 tensor")
            if t.device != q.device:
                raise ValueError(f"{name} is on {t.device}, expected {q.device}")
        if q.dim() != 3 or q.shape[2] != 192:
            raise ValueError("q must be [N, H, 192]")
        n, heads, _ = q.shape
        m = k_rope.shape[0] if k_rope.dim() == 2 else -1
        if k_rope.dim() != 2 or k_rope.shape[1] != 64:
            raise ValueError("k_rope must be [M, 64]")
        if k_nope.shape != (m, heads, 128) or v.shape != (m, heads, 128):
            raise ValueError("k_nope and v must be [M, H, 128], with q's heads and k_rope's tokens")
        if any(t.stride(-1) != 1 for t in (q, k_nope, k_rope, v)):
            raise ValueError("the values of a row of q, k_nope, k_rope and v must be consecutive")
        if len(_EXPANDED_DESCS) > 256:
            _EXPANDED_DESCS.clear()
        d = _EXPANDED_DESCS[key] = ExpandedDesc(
            _int32(batch, "batch"), _int32(heads, "heads"), _int32(n, "query tokens"), _int32(m, "key tokens"),
            int(causal), _stride(q, 0, 192), _stride(q, 1, 192), _stride(k_nope, 0, 128), _stride(k_nope, 1, 128),
            _stride(k_rope, 0, 64), _stride(v, 0, 128), _stride(v, 1, 128))
    return ctypes.byref(d)


def prefill_expanded(q, k_nope, k_rope, v, q_starts, k_starts, causal: bool, sm_scale: float, lse_base: int, out, lse,
                     *, workspace=None, stream=None):
    """mla_prefill_expanded: queries q bf16 [N, H, 192] over keys k_nope bf16
    [M, H, 128] with k_rope bf16 [M, 64] for all heads, and values v bf16
    [M, H, 128]; any strides with rows of consecutive values (parts of a
    projection's output).  Request b's queries and keys are q_starts[b] ..
    q_starts[b + 1] and k_starts[b] .. k_starts[b + 1] (int32 [B + 1] each);
    causal: the last query sees all of them, the one before it one fewer.  out
    bf16 [N, H, 128] and lse fp32 [N, H] are written in place.  The workspace
    is make_prefill_workspace's."""
    lse_base = _int32(lse_base, "lse_base")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("prefill_expanded runs on CUDA tensors only")
    _ints(q_starts, "q_starts", dev, 1)
    _ints(k_starts, "k_starts", dev, 1)
    B = q_starts.numel() - 1
    if B < 0 or k_starts.numel() != B + 1:
        raise ValueError("q_starts and k_starts must be [B + 1]")
    d = _expanded_desc(q, k_nope, k_rope, v, B, bool(causal))
    n, heads, _ = q.shape
    workspace = _prefill_outputs(out, lse, dev, n, heads, 128, workspace, stream, q)
    _launch(load_library().mla_prefill_expanded, dev, stream, q.data_ptr(), k_nope.data_ptr(), k_rope.data_ptr(),
            v.data_ptr(), q_starts.data_ptr(), k_starts.data_ptr(), float(sm_scale), lse_base, out.data_ptr(),
            lse.data_ptr(), d, workspace.data_ptr(), workspace.numel())
    return out, lse


def pages_workspace_size(num_pages: int) -> int:
    n = load_library().mla_pages_workspace_size(_int32(num_pages, "num_pages"))
    if n == 0:
        raise MlaError(-2, "a pool has at least one page")
    return n


def make_pages_workspace(ref_counts) -> torch.Tensor:
    """Scratch for pages_fork, pages_alloc and pages_compact on the pool that
    ref_counts [num_pages] describes; reusable, on the counts' device."""
    return torch.empty(pages_workspace_size(ref_counts.numel()), dtype=torch.uint8,
                       device=ref_counts.device)


def _ints(t, name, device, dim):
    _need(t, name, _I32, device)
    if t.dim() != dim:
        raise ValueError(f"{name} must be {'one' if dim == 1 else 'two'}-dimensional")


_PAGES_DESCS: dict = {}


def _pages_desc(rows, width, pages, page_size, row, kv_dtype):
    """The call's size descriptor (by reference), built once per set of sizes."""
    key = (rows, width, pages, page_size, row, kv_dtype)
    d = _PAGES_DESCS.get(key)
    if d is None:
        if len(_PAGES_DESCS) > 256:
            _PAGES_DESCS.clear()
        d = _PAGES_DESCS[key] = PagesDesc(*(_int32(n, "a size of the pool") for n in key))
    return ctypes.byref(d)


def _pool(kv_pages, name="kv_pages"):
    """Checks a pool; returns its device, shape and dtype code."""
    dev = kv_pages.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    _need(kv_pages, name, _KV_TYPES, dev)
    shape = kv_pages.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [num_pages, 64, 576]")
    return dev, shape, _kv_dtype_code(kv_pages)


def _books(dev, block_table, seq_lens, ref_counts, error_word):
    """Checks a pool's table, lengths and counts; returns (rows, width, pages)."""
    if dev.type != "cuda":
        raise ValueError("the page operations run on CUDA tensors only")
    _ints(block_table, "block_table", dev, 2)
    _ints(ref_counts, "ref_counts", dev, 1)
    rows, width = block_table.shape
    if seq_lens is not None:
        _ints(seq_lens, "seq_lens", dev, 1)
        if seq_lens.numel() != rows:
            raise ValueError("seq_lens must be [num_requests]")
    if error_word is not None:
        _need(error_word, "error_word", _I32, dev)
    return rows, width, ref_counts.numel()


def _opt(t):
    return t.data_ptr() if t is not None else None


def _pages_ws(workspace, ref_counts, stream):
    if workspace is None:
        with _allocating_on(stream, ref_counts.device):
            return make_pages_workspace(ref_counts)
    _need(workspace, "workspace", (torch.uint8,), ref_counts.device)
    return workspace


def pages_copy(src_pages, dst_pages, src, dst, *, error_word=None, stream=None):
    """mla_pages_copy: page src[i] of src_pages to page dst[i] of dst_pages
    (int32 [n] each; two pools of one dtype, or one pool twice)."""
    dev, shape, code = _pool(src_pages, "src_pages")
    _need(dst_pages, "dst_pages", (src_pages.dtype,), dev)
    if dst_pages.dim() != 3 or dst_pages.shape[1:] != shape[1:]:
        raise ValueError("dst_pages must be [num_pages, 64, 576]")
    _ints(src, "src", dev, 1)
    _ints(dst, "dst", dev, 1)
    n = src.numel()
    if dst.numel() != n:
        raise ValueError("src and dst must have the same length")
    if error_word is not None:
        _need(error_word, "error_word", _I32, dev)
    _launch(load_library().mla_pages_copy, dev, stream, src_pages.data_ptr(), dst_pages.data_ptr(),
            src.data_ptr(), dst.data_ptr(), _int32(n, "n"), _int32(dst_pages.shape[0], "dst_num_pages"),
            _pages_desc(0, 1, shape[0], shape[1], shape[2], code), _opt(error_word))
    return dst_pages


def pages_fork(kv_pages, block_table, seq_lens, ref_counts, parents, children, *, workspace=None,
               error_word=None, stream=None):
    """mla_pages_fork: request children[k] becomes a copy of parents[k]
    (int32 [n] each): full pages shared, a partial last page copied.  The
    table [R, W], lengths [R] and counts [num_pages] are updated in place."""
    dev, shape, code = _pool(kv_pages)
    rows, width, pages = _books(dev, block_table, seq_lens, ref_counts, error_word)
    if pages != shape[0]:
        raise ValueError("ref_counts must be [num_pages]")
    _ints(parents, "parents", dev, 1)
    _ints(children, "children", dev, 1)
    n = parents.numel()
    if children.numel() != n:
        raise ValueError("parents and children must have the same length")
    ws = _pages_ws(workspace, ref_counts, stream)
    _launch(load_library().mla_pages_fork, dev, stream, kv_pages.data_ptr(), block_table.data_ptr(),
            seq_lens.data_ptr(), ref_counts.data_ptr(), parents.data_ptr(), children.data_ptr(), _int32(n, "n"),
            _pages_desc(rows, width, pages, shape[1], shape[2], code), ws.data_ptr(), ws.numel(),
            _opt(error_word))


def pages_alloc(block_table, seq_lens, ref_counts, new_lens, *, workspace=None, error_word=None,
                stream=None):
    """mla_pages_alloc: every request gets the pages for new_lens[b] >=
    seq_lens[b] tokens, lowest free pages first (seq_lens is not changed)."""
    dev = block_table.device
    rows, width, pages = _books(dev, block_table, seq_lens, ref_counts, error_word)
    _ints(new_lens, "new_lens", dev, 1)
    if new_lens.numel() != rows:
        raise ValueError("new_lens must be [num_requests]")
    ws = _pages_ws(workspace, ref_counts, stream)
    _launch(load_library().mla_pages_alloc, dev, stream, block_table.data_ptr(), seq_lens.data_ptr(),
            ref_counts.data_ptr(), new_lens.data_ptr(), _pages_desc(rows, width, pages, 64, 576, KV_BF16),
            ws.data_ptr(), ws.numel(), _opt(error_word))


def pages_free(block_table, seq_lens, ref_counts, new_lens, *, window: int = 0, sinks: int = 0,
               error_word=None, stream=None):
    """mla_pages_free: every request is shortened to new_lens[b] tokens (0
    ends it, its own length leaves it) and, with a window, gives up the pages
    that decode_window(window, sinks) no longer sees."""
    window, sinks = _int32(window, "window"), _int32(sinks, "sinks")
    dev = block_table.device
    rows, width, pages = _books(dev, block_table, seq_lens, ref_counts, error_word)
    _ints(new_lens, "new_lens", dev, 1)
    if new_lens.numel() != rows:
        raise ValueError("new_lens must be [num_requests]")
    _launch(load_library().mla_pages_free, dev, stream, block_table.data_ptr(), seq_lens.data_ptr(),
            ref_counts.data_ptr(), new_lens.data_ptr(), window, sinks,
            _pages_desc(rows, width, pages, 64, 576, KV_BF16), _opt(error_word))


def pages_compact(kv_pages, block_table, ref_counts, *, remap=None, workspace=None, error_word=None,
                  stream=None):
    """mla_pages_compact: the live pages move to ids 0 .. live - 1 and the
    table [R, W] and counts follow.  remap: optional int32 [num_pages], each
    page's new id (-1: it was free).  Returns the workspace, whose first two
    int32 words are the number of live pages and of moves."""
    dev, shape, code = _pool(kv_pages)
    rows, width, pages = _books(dev, block_table, None, ref_counts, error_word)
    if pages != shape[0]:
        raise ValueError("ref_counts must be [num_pages]")
    if remap is not None:
        _ints(remap, "remap", dev, 1)
        if remap.numel() != pages:
            raise ValueError("remap must be [num_pages]")
    ws = _pages_ws(workspace, ref_counts, stream)
    _launch(load_library().mla_pages_compact, dev, stream, kv_pages.data_ptr(), block_table.data_ptr(),
            ref_counts.data_ptr(), _opt(remap), _pages_desc(rows, width, pages, shape[1], shape[2], code),
            ws.data_ptr(), ws.numel(), _opt(error_word))
    return ws
