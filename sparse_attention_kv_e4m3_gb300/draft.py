"""Thin Python binding of the operators of a step with drafted tokens in libcsa_index.so
(include/csa_draft.h): norms and rotation of queries and keys, latents normed, rotated and
stored in the paged cache, attention of drafted tokens over it, and the accepted drafts' records moved.

Argument marshalling only, as in `native` and `latent`; there is no fallback. Every tensor is
on the GPU; work goes to `stream`, or the current stream. Outputs and workspaces that
a call makes itself come from that stream's memory; what the caller passes has to be
ready on it, and the caller waits for it before reading results on another one.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import latent, native
from .latent import (LATENT_DIM, CacheArgs, LatentCache, _done, _pick, _same_device, _status, _step, _stream, _want,
                     _workspace, record_bytes)
from .native import _new

ROTATE_MAX_DIM, ROTATE_MAX_ROPE, ROTATE_MAX_HEADS, MAX_WORDS, MAX_REQ, COMMIT_MAX_REQ = 1024, 256, 65536, 16, 65536, 16384
PAIRINGS = {"adjacent": 0, "halves": 1}

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class RotationArgs(ctypes.Structure):
    """Mirror of `csa_rotation`."""
    _fields_ = [("freq", _vp), ("rope_dim", _i32), ("pairing", _i32), ("scale", _f32), ("reserved0", _i32)]


class HeadsArgs(ctypes.Structure):
    """Mirror of `csa_heads`."""
    _fields_ = [("x", _vp), ("out", _vp), ("weight", _vp), ("x_row_stride", _i64), ("x_head_stride", _i64),
                ("out_row_stride", _i64), ("out_head_stride", _i64), ("heads", _i32), ("dim", _i32), ("norm", _i32),
                ("reserved0", _i32)]


class RotateArgs(ctypes.Structure):
    """Mirror of `csa_rotate_args`."""
    _fields_ = [("q", HeadsArgs), ("k", HeadsArgs), ("n", _i64), ("pos", _vp), ("rotation", RotationArgs), ("dtype", _i32),
                ("out_dtype", _i32), ("rope_first", _i32), ("eps", _f32), ("dev_status", _vp)]


class AppendArgs(ctypes.Structure):
    """Mirror of `csa_append_args`."""
    _fields_ = [("cache", CacheArgs), ("x", _vp), ("x_stride", _i64), ("dtype", _i32), ("norm", _i32), ("n", _i64),
                ("slots", _vp), ("pos", _vp), ("rotation", RotationArgs), ("weight", _vp), ("eps", _f32), ("reserved0", _i32),
                ("dev_status", _vp)]


class DraftAttendArgs(ctypes.Structure):
    """Mirror of `csa_draft_attend_args`."""
    _fields_ = [("cache", CacheArgs), ("q", _vp), ("q_row_stride", _i64), ("q_head_stride", _i64), ("num_q", _i32),
                ("num_heads", _i32), ("page_table", _vp), ("num_req", _i32), ("pt_stride", _i32), ("base_len", _vp),
                ("row_start", _vp), ("mask", _vp), ("mask_stride", _i64), ("mask_words", _i32), ("scale", _f32),
                ("out", _vp), ("lse", _vp), ("dev_status", _vp)]


class CommitArgs(ctypes.Structure):
    """Mirror of `csa_commit_args`."""
    _fields_ = [("cache", CacheArgs), ("layer_stride_bytes", _i64), ("num_layers", _i32), ("num_req", _i32),
                ("page_table", _vp), ("pt_stride", _i32), ("path_stride", _i32), ("base_len", _vp), ("draft_len", _vp),
                ("path", _vp), ("path_len", _vp), ("new_len", _vp), ("freed", _vp), ("room", _i64), ("n_freed", _vp),
                ("dev_status", _vp)]


_lib = None


def load():
    """The library with this module's entry points declared. Raises if it has not been built."""
    global _lib
    if _lib is None:
        lib = native.load()
        latent.load()
        P = ctypes.POINTER
        lib.csa_draft_abi_version.argtypes = []
        lib.csa_draft_abi_version.restype = _i32
        lib.csa_head_norm_rotate.argtypes = [P(RotateArgs), _vp]
        lib.csa_head_norm_rotate.restype = ctypes.c_int
        lib.csa_latent_append.argtypes = [P(AppendArgs), _vp]
        lib.csa_latent_append.restype = ctypes.c_int
        lib.csa_draft_attend_workspace_bytes.argtypes = [P(DraftAttendArgs)]
        lib.csa_draft_attend_workspace_bytes.restype = ctypes.c_size_t
        lib.csa_draft_attend.argtypes = [P(DraftAttendArgs), _vp, ctypes.c_size_t, _vp]
        lib.csa_draft_attend.restype = ctypes.c_int
        lib.csa_draft_commit.argtypes = [P(CommitArgs), _vp]
        lib.csa_draft_commit.restype = ctypes.c_int
        _lib = lib
    return _lib


def _dtype(t: torch.dtype, name: str) -> int:
    if t == torch.bfloat16:
        return native.KEYS_BF16
    if t == torch.float32:
        return native.KEYS_F32
    raise TypeError(f"{name} must be float32 or bfloat16")


def _rotation(freq, pairing: str, scale: float, dev) -> RotationArgs:
    kind = PAIRINGS.get(pairing)
    if kind is None:
        raise ValueError(f"pairing: one of {sorted(PAIRINGS)}, not {pairing!r}")
    if freq is None or freq.shape[0] == 0:
        return RotationArgs(None, 0, kind, float(scale), 0)
    if _want(freq, torch.float32, 1, "freq").device != dev:
        raise ValueError(f"freq on {dev}, not on {freq.device}")
    return RotationArgs(freq.data_ptr(), 2 * freq.shape[0], kind, float(scale), 0)


def _weight(w, dim: int, dev, name: str):
    if w is None:
        return None
    if _want(w, torch.float32, 1, name).shape[0] != dim or w.device != dev:
        raise ValueError(f"{name} [{dim}] on {dev}")
    return w.data_ptr()


def _ints(t: torch.Tensor, n: int, dev, name: str) -> int:
    if _want(t, torch.int32, 1, name).shape[0] != n or t.device != dev:
        raise ValueError(f"{name} [{n}] on {dev}, not {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _heads(x: torch.Tensor, weight, norm: bool, out, out_dtype, name: str, stream):
    """One tensor's part of the call: its arguments and its output."""
    _want(x, x.dtype, 3, name)
    dev, (n, heads, dim), (rows, step, _) = x.device, x.shape, x.stride()
    width = heads * dim
    if n == 1 or heads == 1:  # an axis of one element has no stride that matters
        rows, step = (width if n == 1 else rows), (dim if heads == 1 else step)
    if out is None:
        out, out_rows, out_step = _new((n, heads, dim), out_dtype, dev, stream), width, dim
    elif out.shape != x.shape or out.device != dev:
        raise ValueError(f"{name}_out: {tuple(x.shape)} on {dev}, not {tuple(out.shape)} on {out.device}")
    else:
        _want(out, out_dtype, 3, f"{name}_out")
        out_rows, out_step = _step(out, 0, width), _step(out, 1, dim)
    return HeadsArgs(x.data_ptr(), out.data_ptr(), None if weight is None else _weight(weight, dim, dev, f"{name}_weight"), rows, step, out_rows, out_step,
                     heads, dim, 1 if norm else 0, 0), out


def csa_head_norm_rotate(q: torch.Tensor, pos: Optional[torch.Tensor], freq: Optional[torch.Tensor], *, k: Optional[torch.Tensor] = None,
                         q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, q_norm: bool = True,
                         k_norm: bool = True, eps: float = 1e-6, pairing: str = "adjacent", rope_first: bool = False, rope_scale: float = 1.0,
                         q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                         dev_status: Optional[torch.Tensor] = None, stream=None):
    """Norm of every head of q [n, heads, dim] and k [n, k_heads, k_dim] (fp32 or bf16, both the same), and rotation of
    its last (rope_first: first) 2 * len(freq) values to the row's position pos [n] (int32; rows at -1 are left as they are).
    freq None: the norm alone. q_out, k_out: the outputs' memory, or q, k themselves (in place).
    Returns (q_out, k_out), k_out None where k is."""
    dev, n = q.device, q.shape[0]
    if q_out is not None or k_out is not None:
        out_dtype = (k_out if q_out is None else q_out).dtype
    kind, out_kind = _dtype(q.dtype, "q"), _dtype(out_dtype, "the outputs' type")
    qa, q_out = _heads(q, q_weight, q_norm, q_out, out_dtype, "q", stream)
    if k is not None:
        if k.dtype != q.dtype or k.shape[0] != n or k.device != dev:
            raise ValueError(f"k: {n} rows of {q.dtype} on {dev}, as q")
        ka, k_out = _heads(k, k_weight, k_norm, k_out, out_dtype, "k", stream)
    elif k_out is not None:
        raise ValueError("k_out without k")
    else:
        ka = HeadsArgs()
    rotation = _rotation(freq, pairing, rope_scale, dev)
    if pos is None and rotation.rope_dim:
        raise ValueError("pos: a position for every row")
    a = RotateArgs(qa, ka, n, None if pos is None else _ints(pos, n, dev, "pos"), rotation, kind, out_kind, 1 if rope_first else 0, float(eps),
                   _status(dev_status, dev))
    _done(load().csa_head_norm_rotate(ctypes.byref(a), _stream(stream, dev)), "csa_head_norm_rotate")
    return q_out, k_out


def csa_latent_append(x: torch.Tensor, slots: torch.Tensor, pos: Optional[torch.Tensor], cache: LatentCache, freq: Optional[torch.Tensor], *,
                      weight: Optional[torch.Tensor] = None, norm: bool = True, eps: float = 1e-6, pairing: str = "adjacent",
                      rope_scale: float = 1.0, dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Stores rows x [n, 512 + rope] (fp32 or bf16) as the cache's records at `slots` [n] (int64, -1: none), the latent values
    normed (weight [512] fp32, or None for ones), the rope values rotated to pos [n] (int32). pos and freq [rope / 2] are not
    looked at where the cache has no rope values."""
    kind, dev = _dtype(x.dtype, "x"), cache.device
    _want(x, x.dtype, 2, "x")
    _want(slots, torch.int64, 1, "slots")
    _same_device(dev, x, slots)
    n, width = x.shape
    if width != cache.width or slots.shape[0] != n:
        raise ValueError(f"x [n, {cache.width}] and slots [n]")
    if cache.rope_dim:
        if pos is None or freq is None or freq.shape[0] * 2 != cache.rope_dim:
            raise ValueError(f"pos [n] and freq [{cache.rope_dim // 2}]")
    rotation = _rotation(freq if cache.rope_dim else None, pairing, rope_scale, dev)
    a = AppendArgs(cache.args, x.data_ptr(), _step(x, 0, width), kind, 1 if norm else 0, n, slots.data_ptr(),
                   _ints(pos, n, dev, "pos") if cache.rope_dim else None, rotation, _weight(weight, LATENT_DIM, dev, "weight"), float(eps), 0,
                   _status(dev_status, dev))
    _done(load().csa_latent_append(ctypes.byref(a), _stream(stream, dev)), "csa_latent_append")


def csa_draft_attend(q: torch.Tensor, cache: LatentCache, page_table: torch.Tensor, base_len: torch.Tensor, row_start: torch.Tensor, *,
                     scale: float, mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None, stream=None):
    """Latent attention of drafted tokens: row row_start[r] + j of q [num_q, heads, 512 + rope] (bf16) is draft j of request r, whose
    record is at position base_len[r] + j. It sees the base_len[r] records before the drafts and the drafts i whose bit
    i % 64 of word i / 64 of mask [num_q, words] (int64) is set; without a mask those i <= j. Rows of no request are left as they
    are. `ws` is a uint8 workspace of draft_attend_workspace_bytes(...) or more, not in use by another call meanwhile;
    None takes one for the call from torch's allocator. Returns (out [num_q, heads, 512] bf16, lse [num_q, heads] fp32)."""
    _want(q, torch.bfloat16, 3, "q")
    _want(page_table, torch.int32, 2, "page_table", whole=True)
    dev = cache.device
    _same_device(dev, q, page_table)
    n, heads, width = q.shape
    num_req, pt_stride = page_table.shape
    if width != cache.width:
        raise ValueError(f"q [num_q, heads, {cache.width}]")
    mask_ptr, mask_step, words = None, 0, 0
    if mask is not None:
        if _want(mask, torch.int64, 2, "mask").shape[0] != n or mask.device != dev or mask.shape[1] < 1:
            raise ValueError(f"mask [{n}, words] on {dev}, a word at least")
        words = mask.shape[1]
        mask_ptr, mask_step = mask.data_ptr(), _step(mask, 0, words)
    out = _pick(out, (n, heads, LATENT_DIM), torch.bfloat16, dev, "out", stream)
    lse = _pick(lse, (n, heads), torch.float32, dev, "lse", stream)
    a = DraftAttendArgs(cache.args, q.data_ptr(), _step(q, 0, width), _step(q, 1, width), n, heads, page_table.data_ptr(), num_req, pt_stride,
                        _ints(base_len, num_req, dev, "base_len"), _ints(row_start, num_req + 1, dev, "row_start"), mask_ptr, mask_step, words,
                        float(scale), out.data_ptr(), lse.data_ptr(), _status(dev_status, dev))
    lib, ref, st = load(), ctypes.byref(a), _stream(stream, dev)
    if ws is None:
        ws = _workspace(dev, stream, lib.csa_draft_attend_workspace_bytes(ref))
    elif _want(ws, torch.uint8, 1, "ws").device != dev:
        raise ValueError(f"ws is on {ws.device}, not on {dev}")
    _done(lib.csa_draft_attend(ref, ws.data_ptr(), ws.shape[0], st), "csa_draft_attend")
    return out, lse


def draft_attend_workspace_bytes(num_q: int, heads: int, num_req: int, pt_stride: int) -> int:
    """Workspace of csa_draft_attend for these sizes."""
    a = DraftAttendArgs(num_q=int(num_q), num_heads=int(heads), num_req=int(num_req), pt_stride=int(pt_stride))
    return int(load().csa_draft_attend_workspace_bytes(ctypes.byref(a)))


class LayeredCache:
    """The latent caches of every layer, with one page table: `pages` uint8 [layers, num_pages, >= 64 * record bytes]."""

    def __init__(self, pages: torch.Tensor, rope_dim: int = 64, record_format="bf16"):
        _want(pages, torch.uint8, 3, "pages")
        self.pages, self.device, self.rope_dim, self.record_format = pages, pages.device, int(rope_dim), record_format
        self.layers = [LatentCache(p, rope_dim, record_format) for p in pages]
        if not self.layers:
            raise ValueError("pages of at least one layer")
        self.args, self.layer_stride = self.layers[0].args, _step(pages, 0, pages.shape[1] * pages.shape[2])

    @staticmethod
    def empty(layers: int, num_pages: int, rope_dim: int = 64, record_format="bf16", device="cuda") -> "LayeredCache":
        n = native.PAGE_RECORDS * record_bytes(record_format, rope_dim)
        return LayeredCache(torch.empty((layers, num_pages, n), dtype=torch.uint8, device=device), rope_dim, record_format)


class Committed(NamedTuple):
    """What csa_draft_commit makes beside the moved records."""
    new_len: torch.Tensor  # [num_req] int32
    freed: torch.Tensor    # [room] int32, -1 past the last
    n_freed: torch.Tensor  # [1] int32


def csa_draft_commit(cache, page_table: torch.Tensor, base_len: torch.Tensor, draft_len: torch.Tensor, path: torch.Tensor,
                     path_len: torch.Tensor, *, room: Optional[int] = None, out: Optional[Committed] = None,
                     dev_status: Optional[torch.Tensor] = None, stream=None) -> Committed:
    """The end of a step: request r's accepted drafts path[r][0] < path[r][1] < ... (path_len[r] of the draft_len[r] behind its
    base_len[r] records) move to the front, in `cache` (a LatentCache, or a LayeredCache for every layer's at once), and the pages
    behind the new lengths are listed. `room`: entries for them (as many as the table has, where it is not given)."""
    layers = cache.layers if isinstance(cache, LayeredCache) else [cache]
    dev = cache.device
    _want(page_table, torch.int32, 2, "page_table", whole=True)
    _want(path, torch.int32, 2, "path", whole=True)
    _same_device(dev, page_table, path)
    num_req, pt_stride = page_table.shape
    if path.shape[0] != num_req:
        raise ValueError("path [num_req, most]")
    if out is None:
        room = num_req * pt_stride if room is None else int(room)
        if room < 0:
            raise ValueError("room: at least 0")
        buf = _new((num_req + room + 1,), torch.int32, dev, stream)
        out = Committed(*torch.unsafe_split_with_sizes(buf, (num_req, room, 1)))
    else:
        room = out.freed.shape[0] if room is None else int(room)
        for t, size, name in zip(out, (num_req, room, 1), Committed._fields):
            _pick(t, (size,), torch.int32, dev, name, stream)
    a = CommitArgs(cache.args, cache.layer_stride if len(layers) > 1 else 0, len(layers), num_req, page_table.data_ptr(), pt_stride,
                   path.shape[1], _ints(base_len, num_req, dev, "base_len"), _ints(draft_len, num_req, dev, "draft_len"),
                   path.data_ptr(), _ints(path_len, num_req, dev, "path_len"), out.new_len.data_ptr(), out.freed.data_ptr(), room,
                   out.n_freed.data_ptr(), _status(dev_status, dev))
    _done(load().csa_draft_commit(ctypes.byref(a), _stream(stream, dev)), "csa_draft_commit")
    return out
