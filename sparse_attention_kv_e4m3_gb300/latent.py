"""Thin Python binding of the latent-cache operators of libcsa_index.so
(include/csa_latent.h): block tables, the paged latent cache's writer and reader,
and latent attention, absorbed (over the cache) and expanded (prompts).

Argument marshalling only, as in `native`; there is no fallback. Every tensor is
on the GPU; work goes to `stream`, or the current stream. Outputs and workspaces that
a call makes itself come from that stream's memory; what the caller passes has to be
ready on it, and the caller waits for it before reading results on another one.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import native
from .native import CSA_OK, _check, _empty, _new

LATENT_DIM, MAX_HEADS, TABLES_MAX_REQ = 512, 128, 16384
PREFILL_NOPE, PREFILL_ROPE, PREFILL_V = 128, 64, 128
FORMAT_BF16, FORMAT_MXFP4 = 0, 1
FORMATS = {"bf16": FORMAT_BF16, "mxfp4": FORMAT_MXFP4, FORMAT_BF16: FORMAT_BF16, FORMAT_MXFP4: FORMAT_MXFP4}
DEV_POOL, DEV_ROWS = 64, 128

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class CacheArgs(ctypes.Structure):
    """Mirror of `csa_latent_cache`."""
    _fields_ = [("pages", _vp), ("num_pages", _i64), ("page_stride_bytes", _i64), ("rope_dim", _i32),
                ("record_format", _i32)]


class TablesArgs(ctypes.Structure):
    """Mirror of `csa_tables_args`."""
    _fields_ = [("old_len", _vp), ("new_len", _vp), ("num_req", _i32), ("pt_stride", _i32), ("page_table", _vp),
                ("free_pages", _vp), ("n_free", _i64), ("n_rows", _i64), ("row_req", _vp), ("row_pos", _vp),
                ("row_len", _vp), ("row_slot", _vp), ("row_start", _vp), ("kv_start", _vp), ("taken", _vp),
                ("dev_status", _vp)]


class LatentWriteArgs(ctypes.Structure):
    """Mirror of `csa_latent_write_args`."""
    _fields_ = [("cache", CacheArgs), ("x", _vp), ("x_stride", _i64), ("dtype", _i32), ("reserved0", _i32),
                ("n", _i64), ("slots", _vp), ("dev_status", _vp)]


class LatentReadArgs(ctypes.Structure):
    """Mirror of `csa_latent_read_args`."""
    _fields_ = [("cache", CacheArgs), ("page_table", _vp), ("num_req", _i32), ("pt_stride", _i32),
                ("kv_start", _vp), ("n_rows", _i64), ("out", _vp), ("dev_status", _vp)]


class AttendArgs(ctypes.Structure):
    """Mirror of `csa_latent_attend_args`."""
    _fields_ = [("cache", CacheArgs), ("q", _vp), ("q_row_stride", _i64), ("q_head_stride", _i64), ("num_q", _i32),
                ("num_heads", _i32), ("page_table", _vp), ("num_req", _i32), ("pt_stride", _i32), ("row_req", _vp),
                ("row_len", _vp), ("idx", _vp), ("idx_stride", _i64), ("top", _i32), ("scale", _f32), ("out", _vp),
                ("lse", _vp), ("dev_status", _vp)]


class PrefillArgs(ctypes.Structure):
    """Mirror of `csa_latent_prefill_args`."""
    _fields_ = [("q", _vp), ("k_nope", _vp), ("k_rope", _vp), ("v", _vp), ("q_row_stride", _i64),
                ("q_head_stride", _i64), ("k_row_stride", _i64), ("k_head_stride", _i64), ("rope_row_stride", _i64),
                ("v_row_stride", _i64), ("v_head_stride", _i64), ("total_q", _i64), ("total_k", _i64),
                ("q_start", _vp), ("kv_start", _vp), ("num_req", _i32), ("num_heads", _i32), ("causal", _i32),
                ("scale", _f32), ("out", _vp), ("lse", _vp), ("dev_status", _vp)]


_lib = None


def load():
    """The library with this module's entry points declared. Raises if it has not been built."""
    global _lib
    if _lib is None:
        lib = native.load()
        P = ctypes.POINTER
        lib.csa_latent_abi_version.argtypes = []
        lib.csa_latent_abi_version.restype = _i32
        lib.csa_latent_record_bytes.argtypes = [_i32, _i32]
        lib.csa_latent_record_bytes.restype = _i64
        lib.csa_build_tables.argtypes = [P(TablesArgs), _vp]
        lib.csa_build_tables.restype = ctypes.c_int
        lib.csa_latent_write.argtypes = [P(LatentWriteArgs), _vp]
        lib.csa_latent_write.restype = ctypes.c_int
        lib.csa_latent_read.argtypes = [P(LatentReadArgs), _vp]
        lib.csa_latent_read.restype = ctypes.c_int
        lib.csa_latent_attend_workspace_bytes.argtypes = [P(AttendArgs)]
        lib.csa_latent_attend_workspace_bytes.restype = ctypes.c_size_t
        lib.csa_latent_attend.argtypes = [P(AttendArgs), _vp, ctypes.c_size_t, _vp]
        lib.csa_latent_attend.restype = ctypes.c_int
        lib.csa_latent_prefill.argtypes = [P(PrefillArgs), _vp]
        lib.csa_latent_prefill.restype = ctypes.c_int
        _lib = lib
    return _lib


def record_bytes(record_format, rope_dim: int) -> int:
    """Bytes of one record; raises for a format or rope_dim that the cache does not have."""
    n = int(load().csa_latent_record_bytes(FORMATS.get(record_format, -1), int(rope_dim)))
    if n == 0:
        raise ValueError(f"no latent record of format {record_format!r} with rope_dim {rope_dim}")
    return n


def _want(t: torch.Tensor, dtype, dims: int, name: str, whole: bool = False) -> torch.Tensor:
    """Checks a tensor argument: on the GPU, of this type and rank, contiguous in its last axis (or `whole`)."""
    if not (t.is_cuda and t.dtype == dtype and t.dim() == dims):
        raise ValueError(f"{name}: a {dims}-d {dtype} CUDA tensor, not {tuple(t.shape)} {t.dtype} on {t.device}")
    if not t.is_contiguous() and (whole or (t.stride(-1) != 1 and t.shape[-1] != 1)):
        raise ValueError(f"{name}: contiguous{'' if whole else ' in its last axis'}")
    return t


def _pick(out, shape, dtype, device, name, stream):
    """The caller's output tensor, checked, or a new one."""
    if out is None:
        return _new(shape, dtype, device, stream)
    _want(out, dtype, len(shape), name, whole=True)
    if out.shape != shape or out.device != device:
        raise ValueError(f"{name}: {tuple(shape)} on {device}, not {tuple(out.shape)} on {out.device}")
    return out


def _status(t, device):
    if t is None:
        return None
    if _want(t, torch.int32, 1, "dev_status").device != device or t.shape[0] < 1:
        raise ValueError(f"dev_status: one int32 on {device}")
    return t.data_ptr()


def _stream(stream, device) -> int:
    """The given stream, or the current one, as an address. The library launches on the current device, so the tensors
    and the stream have to be there."""
    if device.index != torch._C._cuda_getDevice() or (stream is not None and stream.device != device):
        where = "" if stream is None else f", the stream on {stream.device}"
        raise ValueError(f"tensors on {device}, the current device is cuda:{torch._C._cuda_getDevice()}{where}")
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _done(st: int, what: str) -> None:
    if st != CSA_OK:
        _check(st, what)


def _step(t: torch.Tensor, dim: int, width: int) -> int:
    """The stride along `dim`; an axis of one element has none that matters."""
    return t.stride(dim) if t.shape[dim] > 1 else width


def _same_device(device, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"every tensor is on {device}, not on {t.device}")


class LatentCache:
    """A paged latent cache: `pages` uint8 [num_pages, >= 64 * record bytes], rows page stride apart."""

    def __init__(self, pages: torch.Tensor, rope_dim: int = 64, record_format="bf16"):
        _want(pages, torch.uint8, 2, "pages")
        self.record_format, self.rope_dim = FORMATS.get(record_format, -1), int(rope_dim)
        self.record_bytes = record_bytes(record_format, rope_dim)
        if pages.shape[1] < native.PAGE_RECORDS * self.record_bytes:
            raise ValueError(f"pages hold at least {native.PAGE_RECORDS * self.record_bytes} bytes")
        self.pages, self.device = pages, pages.device
        self.width = LATENT_DIM + self.rope_dim
        self.args = CacheArgs(pages.data_ptr(), pages.shape[0], _step(pages, 0, pages.shape[1]), self.rope_dim, self.record_format)

    @staticmethod
    def empty(num_pages: int, rope_dim: int = 64, record_format="bf16", device="cuda") -> "LatentCache":
        n = native.PAGE_RECORDS * record_bytes(record_format, rope_dim)
        return LatentCache(torch.empty((num_pages, n), dtype=torch.uint8, device=device), rope_dim, record_format)


class StepTables(NamedTuple):
    """What csa_build_tables makes beside the page table."""
    row_req: torch.Tensor    # [n_rows] int32
    row_pos: torch.Tensor    # [n_rows] int32
    row_len: torch.Tensor    # [n_rows] int32
    row_slot: torch.Tensor   # [n_rows] int64
    row_start: torch.Tensor  # [num_req + 1] int32
    kv_start: torch.Tensor   # [num_req + 1] int32
    taken: torch.Tensor      # [1] int32


def empty_tables(num_req: int, n_rows: int, device="cuda", stream=None) -> StepTables:
    """Tables for csa_build_tables to fill (on `stream`, or the current stream), in one allocation."""
    buf = _new((5 * n_rows + 2 * num_req + 3,), torch.int32, device, stream)
    slot, req, pos, length, row_start, kv_start, taken = torch.unsafe_split_with_sizes(
        buf, (2 * n_rows, n_rows, n_rows, n_rows, num_req + 1, num_req + 1, 1))
    return StepTables(req, pos, length, slot.view(torch.int64), row_start, kv_start, taken)


def csa_build_tables(old_len: torch.Tensor, new_len: torch.Tensor, page_table: torch.Tensor, free_pages: torch.Tensor,
                     n_rows: int, out: Optional[StepTables] = None, dev_status: Optional[torch.Tensor] = None,
                     stream=None) -> StepTables:
    """Block tables and slot maps of one step: request r holds old_len[r] records and gets new_len[r]
    more. page_table [num_req, pt_stride] gets the new pages in place, out of free_pages; the maps of
    the new records, one row each (n_rows of them, the rest padding), are returned."""
    _want(old_len, torch.int32, 1, "old_len")
    _want(new_len, torch.int32, 1, "new_len")
    _want(page_table, torch.int32, 2, "page_table", whole=True)
    _want(free_pages, torch.int32, 1, "free_pages")
    dev, n, n_rows = old_len.device, old_len.shape[0], int(n_rows)
    _same_device(dev, new_len, page_table, free_pages)
    if new_len.shape[0] != n or page_table.shape[0] != n or n_rows < 0:
        raise ValueError("old_len, new_len and page_table: one row a request; n_rows at least 0")
    if out is None:
        out = empty_tables(n, n_rows, dev, stream)
        # one allocation: slots, three maps, two running sums (never empty, as the maps may be), the count
        start = out.row_start.data_ptr()
        at = start - 20 * n_rows
        req, pos, length = at + 8 * n_rows, at + 12 * n_rows, at + 16 * n_rows
        ptrs = (req, pos, length, at, start, start + 4 * (n + 1), start + 8 * (n + 1))
    else:
        for t, (size, dtype), name in zip(out, [(n_rows, torch.int32)] * 3 + [(n_rows, torch.int64)] +
                                          [(n + 1, torch.int32)] * 2 + [(1, torch.int32)], StepTables._fields):
            _pick(t, (size,), dtype, dev, name, stream)
        ptrs = tuple(t.data_ptr() for t in out)
    a = TablesArgs(old_len.data_ptr(), new_len.data_ptr(), n, page_table.shape[1], page_table.data_ptr(),
                   free_pages.data_ptr(), free_pages.shape[0], n_rows, *ptrs, _status(dev_status, dev))
    _done(load().csa_build_tables(ctypes.byref(a), _stream(stream, dev)), "csa_build_tables")
    return out


def csa_latent_write(x: torch.Tensor, slots: torch.Tensor, cache: LatentCache,
                     dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Stores rows x [n, 512 + rope] (fp32 or bf16) as the cache's records at `slots` [n] (int64)."""
    dtype, dev = x.dtype, cache.device
    if dtype != torch.bfloat16 and dtype != torch.float32:
        raise TypeError("x must be float32 or bfloat16")
    _want(x, dtype, 2, "x")
    _want(slots, torch.int64, 1, "slots")
    _same_device(dev, x, slots)
    n, width = x.shape
    if width != cache.width or slots.shape[0] != n:
        raise ValueError(f"x [n, {cache.width}] and slots [n]")
    a = LatentWriteArgs(cache.args, x.data_ptr(), _step(x, 0, width),
                        native.KEYS_BF16 if dtype == torch.bfloat16 else native.KEYS_F32, 0, n, slots.data_ptr(),
                        _status(dev_status, dev))
    _done(load().csa_latent_write(ctypes.byref(a), _stream(stream, dev)), "csa_latent_write")


def csa_latent_read(cache: LatentCache, page_table: torch.Tensor, kv_start: torch.Tensor, n_rows: int,
                    out: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Histories as rows [n_rows, 512 + rope] in bf16: record j of request r at kv_start[r] + j.
    Rows that no request covers are left as they are (whatever was there, where `out` is not given)."""
    _want(page_table, torch.int32, 2, "page_table", whole=True)
    _want(kv_start, torch.int32, 1, "kv_start")
    dev, n_rows = cache.device, int(n_rows)
    _same_device(dev, page_table, kv_start)
    num_req, width = page_table.shape
    if kv_start.shape[0] != num_req + 1 or n_rows < 0:
        raise ValueError("page_table [num_req, pt_stride], kv_start [num_req + 1], n_rows at least 0")
    out = _pick(out, (n_rows, cache.width), torch.bfloat16, dev, "out", stream)
    a = LatentReadArgs(cache.args, page_table.data_ptr(), num_req, width, kv_start.data_ptr(), n_rows, out.data_ptr(),
                       _status(dev_status, dev))
    _done(load().csa_latent_read(ctypes.byref(a), _stream(stream, dev)), "csa_latent_read")
    return out


def _workspace(device, stream, size: int) -> torch.Tensor:
    """A call's own workspace of at least `size` bytes. None is kept for the next call: a call is two launches, and
    another host thread's call on the same stream may be enqueued between them."""
    return _empty(max(size, 16), torch.uint8, device, stream)


def csa_latent_attend(q: torch.Tensor, cache: LatentCache, page_table: torch.Tensor, row_len: torch.Tensor, *,
                      scale: float, idx: Optional[torch.Tensor] = None, row_req: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None, stream=None):
    """Latent attention, absorbed form: q [num_q, heads, 512 + rope] bf16 over the records below row_len[b]
    of request row_req[b] (identity when None), or over the positions idx [num_q, top] (-1: none; top
    may be 0) among them. `ws` is a uint8 workspace of attend_workspace_bytes(...) or more, not in use by another call
    meanwhile; None takes one for the call (42 MB at most) from torch's allocator.
    Returns (out [num_q, heads, 512] bf16, lse [num_q, heads] fp32)."""
    _want(q, torch.bfloat16, 3, "q")
    _want(page_table, torch.int32, 2, "page_table", whole=True)
    _want(row_len, torch.int32, 1, "row_len")
    dev = cache.device
    _same_device(dev, q, page_table, row_len, idx, row_req)
    n, heads, width = q.shape
    num_req, pt_stride = page_table.shape
    if width != cache.width or row_len.shape[0] != n:
        raise ValueError(f"q [num_q, heads, {cache.width}], row_len [num_q]")
    idx_ptr, idx_step, top, req_ptr = None, 0, 0, None
    if idx is not None:
        if _want(idx, torch.int32, 2, "idx").shape[0] != n:
            raise ValueError("idx [num_q, top]")
        if idx.shape[1] == 0:  # its address is null, which the library reads as whole histories: nothing is listed instead
            idx = _empty((n, 1), torch.int32, dev, stream, -1)
        top = idx.shape[1]
        idx_ptr, idx_step = idx.data_ptr(), _step(idx, 0, top)
    if row_req is not None:
        if _want(row_req, torch.int32, 1, "row_req").shape[0] != n:
            raise ValueError("row_req [num_q]")
        req_ptr = row_req.data_ptr()
    out = _pick(out, (n, heads, LATENT_DIM), torch.bfloat16, dev, "out", stream)
    lse = _pick(lse, (n, heads), torch.float32, dev, "lse", stream)
    a = AttendArgs(cache.args, q.data_ptr(), _step(q, 0, width), _step(q, 1, width), n, heads, page_table.data_ptr(),
                   num_req, pt_stride, req_ptr, row_len.data_ptr(), idx_ptr, idx_step, top, float(scale),
                   out.data_ptr(), lse.data_ptr(), _status(dev_status, dev))
    lib, ref, st = load(), ctypes.byref(a), _stream(stream, dev)
    if ws is None:
        ws = _workspace(dev, stream, lib.csa_latent_attend_workspace_bytes(ref))
    elif _want(ws, torch.uint8, 1, "ws").device != dev:
        raise ValueError(f"ws is on {ws.device}, not on {dev}")
    _done(lib.csa_latent_attend(ref, ws.data_ptr(), ws.shape[0], st), "csa_latent_attend")
    return out, lse


def attend_workspace_bytes(num_q: int, heads: int, pt_stride: int, top: int = 0) -> int:
    """Workspace of csa_latent_attend for these sizes (top: positions a row, 0 for whole histories)."""
    a = AttendArgs(num_q=int(num_q), num_heads=int(heads), pt_stride=int(pt_stride), top=int(top), idx=16 if top else None)
    return int(load().csa_latent_attend_workspace_bytes(ctypes.byref(a)))


def csa_latent_prefill(q: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor,
                       q_start: torch.Tensor, kv_start: torch.Tensor, *, scale: float, causal: bool = True,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       dev_status: Optional[torch.Tensor] = None, stream=None):
    """Latent attention, expanded form: q [total_q, heads, 192], k_nope and v [total_k, heads, 128], k_rope
    [total_k, 64], all bf16; request r has rows q_start[r] .. q_start[r + 1] of q and kv_start[r] ..
    kv_start[r + 1] of the keys. Rows of no request are left as they are. Returns (out [total_q, heads, 128] bf16, lse [total_q, heads] fp32)."""
    _want(q, torch.bfloat16, 3, "q")
    _want(k_nope, torch.bfloat16, 3, "k_nope")
    _want(v, torch.bfloat16, 3, "v")
    _want(k_rope, torch.bfloat16, 2, "k_rope")
    _want(q_start, torch.int32, 1, "q_start")
    _want(kv_start, torch.int32, 1, "kv_start")
    dev = q.device
    _same_device(dev, k_nope, k_rope, v, q_start, kv_start)
    tq, heads, width = q.shape
    tk = k_nope.shape[0]
    if (width != PREFILL_NOPE + PREFILL_ROPE or k_nope.shape != (tk, heads, PREFILL_NOPE) or
            v.shape != (tk, heads, PREFILL_V) or k_rope.shape != (tk, PREFILL_ROPE) or
            q_start.shape != kv_start.shape or q_start.shape[0] < 1):
        raise ValueError("q [tq, h, 192], k_nope and v [tk, h, 128], k_rope [tk, 64], q_start and kv_start [num_req + 1]")
    out = _pick(out, (tq, heads, PREFILL_V), torch.bfloat16, dev, "out", stream)
    lse = _pick(lse, (tq, heads), torch.float32, dev, "lse", stream)
    a = PrefillArgs(q.data_ptr(), k_nope.data_ptr(), k_rope.data_ptr(), v.data_ptr(), _step(q, 0, width),
                    _step(q, 1, width), _step(k_nope, 0, 128), _step(k_nope, 1, 128), _step(k_rope, 0, 64),
                    _step(v, 0, 128), _step(v, 1, 128), tq, tk, q_start.data_ptr(), kv_start.data_ptr(),
                    q_start.shape[0] - 1, heads, 1 if causal else 0, float(scale), out.data_ptr(), lse.data_ptr(),
                    _status(dev_status, dev))
    _done(load().csa_latent_prefill(ctypes.byref(a), _stream(stream, dev)), "csa_latent_prefill")
    return out, lse
