"""Thin Python binding of include/splitzip_pages.h: a KV cache in pages, in BF16,
FP8 E5M2 or quantised to 8 or 4 bits (the store that fills it, the load that reads
sequences back out of it, the attention of a batch's new tokens over it).

Argument marshalling only, as in ``serving``: PyTorch supplies device memory and
streams, nothing is allocated or synchronised by a call, and what the C ABI cannot
see (shapes, types, the extent of every buffer) is checked here (``SplitZipError``
with ``ERR_INVALID_ARG``).

A pool is a ``Pages``: keys and values [pages, page_tokens, kv_heads, row], in any
strides with contiguous rows, and for the quantised formats their exponent bytes
[pages, page_tokens, kv_heads, 4].  ``alloc_pages`` makes one whose pages lie head by
head.  ``splitzip_qk_norm_rope`` fills pages of BF16 and E5M2 too: its slots count
token strides of the pool, ``page * (k.stride(0) // k.stride(1)) + slot``.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import splitzip as _sz
from .serving import _MOST, _VIEW, View, _bad, _bf16, _check, _check_array, _check_view, _current_device, _stream_of
from .splitzip import SplitZipError  # noqa: F401  (raised by the checks)

BF16, E5M2, INT8, E2M1 = 0, 1, 2, 3
_FORMAT = {torch.bfloat16: BF16, torch.float8_e5m2: E5M2, torch.int8: INT8, torch.uint8: E2M1}
_DTYPE = {"bf16": torch.bfloat16, "e5m2": torch.float8_e5m2, "int8": torch.int8, "e2m1": torch.uint8}
_MOST_TOKENS = (1 << 31) - 256     # of a sequence that attention takes
_u32, _i64, _f32, _vp = ctypes.c_uint32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class PageRows(ctypes.Structure):
    _fields_ = [("data", _vp), ("stride_p", _i64), ("stride_t", _i64), ("stride_h", _i64),
                ("exponents", _vp), ("exp_stride_p", _i64), ("exp_stride_t", _i64), ("exp_stride_h", _i64)]


class Pool(ctypes.Structure):
    _fields_ = [("k", PageRows), ("v", PageRows), ("pages", _u32), ("page_tokens", _u32), ("kv_heads", _u32),
                ("head_dim", _u32), ("format", _u32)]


class PagesStoreArgs(ctypes.Structure):
    _fields_ = [("k", View), ("v", View), ("slots", _vp), ("pool", Pool), ("n", _u32)]


class PagesLoadArgs(ctypes.Structure):
    _fields_ = [("pool", Pool), ("table", _vp), ("lens", _vp), ("k_out", View), ("v_out", View),
                ("batch", _u32), ("tokens", _u32), ("table_width", _u32), ("out_format", _u32)]


class PagedAttentionArgs(ctypes.Structure):
    _fields_ = [("q", View), ("out", View), ("pool", Pool), ("lse", _vp), ("table", _vp), ("q_start", _vp), ("lens", _vp),
                ("batch", _u32), ("tokens", _u32), ("max_q_tokens", _u32), ("kv_tokens", _u32), ("table_width", _u32),
                ("q_heads", _u32), ("window", _u32), ("sinks", _u32), ("scale", _f32)]


# The structures as packed bytes, as in ``serving``; a pool's are packed once, in its handle.
_POOL_BYTES = ctypes.sizeof(Pool)
_POOL = struct.Struct("@" + 2 * "P3qP3q" + "5I4x")
_STORE = struct.Struct(f"@{2 * _VIEW}P{_POOL_BYTES}sI4x")
_LOAD = struct.Struct(f"@{_POOL_BYTES}s2P{2 * _VIEW}4I")
_ATTENTION = struct.Struct(f"@{2 * _VIEW}{_POOL_BYTES}s4P8If4x")

_lib = None
_fn_store = _fn_load = _fn_attention = None
_B16, _F8, _F32, _I32, _I64, _U8 = (torch.bfloat16, torch.float8_e5m2, torch.float32, torch.int32, torch.int64, torch.uint8)


def library() -> ctypes.CDLL:
    """libsplitzip.so with the signatures of splitzip_pages.h (raises if it has not been built)."""
    global _lib, _fn_store, _fn_load, _fn_attention
    if _lib is None:
        lib = _sz.library()
        sig = {
            "splitzip_pages_store": (ctypes.c_int, [_vp, _vp]),
            "splitzip_pages_load": (ctypes.c_int, [_vp, _vp]),
            "splitzip_paged_attention_workspace_bytes": (ctypes.c_size_t, [_vp]),
            "splitzip_paged_attention": (ctypes.c_int, [_vp, _vp, ctypes.c_size_t, _vp]),
            "splitzip_paged_attention_test": (ctypes.c_int, [_vp, _vp, ctypes.c_size_t, _vp, _vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
        _fn_store, _fn_load, _fn_attention = lib.splitzip_pages_store, lib.splitzip_pages_load, lib.splitzip_paged_attention
    return _lib


class Pages:
    """A pool of pages: k, v [pages, page_tokens, kv_heads, row] of torch.bfloat16, torch.float8_e5m2, torch.int8
    (row = head_dim) or torch.uint8 (two E2M1 codes to a byte, row = head_dim / 2); k_exp, v_exp uint8
    [pages, page_tokens, kv_heads, 4] for the last two.  The handle keeps views of them, and addresses: a call whose
    pool's memory has been resized since is refused."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_exp: torch.Tensor | None = None,
                 v_exp: torch.Tensor | None = None):
        fmt = _FORMAT.get(k.dtype)
        if fmt is None:
            _bad(f"pages are BF16, E5M2, int8 or uint8 (E2M1), not {k.dtype}")
        if v.dtype != k.dtype:
            _bad(f"keys are {k.dtype}, values {v.dtype}")
        if k.dim() != 4:
            _bad("pages are [pages, page_tokens, kv_heads, row]")
        shape = tuple(k.shape)
        _check_view(k, shape, "k")
        _check_view(v, shape, "v")
        if fmt in (INT8, E2M1):
            if k_exp is None or v_exp is None:
                _bad("quantised pages need exponent bytes")
            for t, what in ((k_exp, "k_exp"), (v_exp, "v_exp")):
                if t.dtype != _U8:
                    _bad(f"{what} is {t.dtype}, torch.uint8 needed")
                _check_view(t, (*shape[:3], 4), what)
        elif k_exp is not None or v_exp is not None:
            _bad("exponent bytes belong to quantised pages")
        for t in (v, k_exp, v_exp):
            if t is not None and t.device != k.device:
                _bad("a pool lies on one device")
        # Views of its own, which a caller's k.resize_() or k.set_() does not change.
        self._tensors = tuple(None if t is None else t.detach() for t in (k, v, k_exp, v_exp))
        self._now = tuple(t.data_ptr for t in self._tensors if t is not None)     # where they are, asked with each call
        self._then = tuple(f() for f in self._now)
        self.format, self.pages, self.page_tokens, self.kv_heads = fmt, *shape[:3]
        self.head_dim = 2 * shape[3] if fmt == E2M1 else shape[3]
        self.device, self.index = k.device, k.get_device()
        rows = []
        for t, e in ((k, k_exp), (v, v_exp)):
            rows += [t.data_ptr(), *t.stride()[:3], *((0, 0, 0, 0) if e is None else (e.data_ptr(), *e.stride()[:3]))]
        self._packed = _POOL.pack(*rows, *shape[:3], self.head_dim, fmt)

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_exp = property(lambda self: self._tensors[2])
    v_exp = property(lambda self: self._tensors[3])

    @property
    def packed(self) -> bytes:
        """The pool as the library takes it."""
        now, then = self._now, self._then
        if now[0]() != then[0] or now[1]() != then[1] or (len(now) > 2 and (now[2]() != then[2] or now[3]() != then[3])):
            _bad("the pool's memory has moved since its handle was made")
        return self._packed


def alloc_pages(pages: int, page_tokens: int, kv_heads: int, head_dim: int, fmt: str = "bf16", device="cuda") -> Pages:
    """A pool of zeros of this format ("bf16", "e5m2", "int8" or "e2m1"), a page's rows head by head."""
    if fmt not in _DTYPE:
        _bad(f"no format {fmt!r}")
    row = head_dim // 2 if fmt == "e2m1" else head_dim

    def zeros(width, dtype):
        return torch.zeros((pages, kv_heads, page_tokens, width), dtype=dtype, device=device).transpose(1, 2)
    exps = [zeros(4, _U8) if fmt in ("int8", "e2m1") else None for _ in range(2)]
    return Pages(zeros(row, _DTYPE[fmt]), zeros(row, _DTYPE[fmt]), *exps)


def _check_device(pages: Pages, *tensors):
    """The pool, the rows that go with it and the call are on one device: a stream reaches no other."""
    for t in (pages.k, *tensors):
        if t is not None and t.get_device() != _current_device():
            _bad(f"a tensor on {t.device}, the current device is cuda:{_current_device()}")


# ------------------------------------------------------------------ store

def splitzip_pages_store(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, pages: Pages, stream=None):
    """Write k, v (BF16 [n, kv_heads, head_dim]) to their slots (int64 [n], page * page_tokens + slot) of the pool;
    asynchronous.  A token whose slot is outside the pool is dropped."""
    ks = k.shape
    kst, vst = k.stride(), v.stride()
    ok = (len(ks) == 3 and ks[1] == pages.kv_heads and ks[2] == pages.head_dim and v.shape == ks
          and k.dtype is _B16 and v.dtype is _B16 and kst[2] == 1 and vst[2] == 1 and k.get_device() == v.get_device() == pages.index == _current_device()
          and slots.dtype is _I64 and slots.shape == ks[:1] and slots.is_contiguous() and slots.get_device() == pages.index)
    if not ok:
        _bf16(k, "k")
        _bf16(v, "v")
        shape = (ks[0] if ks else 0, pages.kv_heads, pages.head_dim)
        _check_view(k, shape, "k")
        _check_view(v, shape, "v")
        _check_array(slots, _I64, shape[:1], "slots")
        _check_device(pages, k, v, slots)
        _bad("these arguments are not accepted")
    a = _STORE.pack(k.data_ptr(), 0, kst[0], kst[1], v.data_ptr(), 0, vst[0], vst[1], slots.data_ptr(), pages.packed, ks[0])
    if _fn_store is None:
        library()
    status = _fn_store(a, _stream_of(stream))
    if status:
        _check(status, "splitzip_pages_store")


# ------------------------------------------------------------------- load

def splitzip_pages_load(pages: Pages, table: torch.Tensor, lens: torch.Tensor | None, k_out: torch.Tensor,
                        v_out: torch.Tensor, stream=None):
    """Read the first lens[b] (int32 [batch]; None: all) tokens of every sequence out of the pages that table
    (int32 [batch, width]) names, into k_out and v_out [batch, tokens, kv_heads, head_dim] (BF16, or E5M2 from a
    pool of E5M2); asynchronous.  Rows behind a sequence's length stay as they were."""
    ks, ts, kind = k_out.shape, table.shape, k_out.dtype
    kst, vst = k_out.stride(), v_out.stride()
    ok = (len(ks) == 4 and ks[2] == pages.kv_heads and ks[3] == pages.head_dim and v_out.shape == ks and v_out.dtype is kind
          and (kind is _B16 or (kind is _F8 and pages.format == E5M2)) and kst[3] == 1 and vst[3] == 1
          and k_out.get_device() == v_out.get_device() == pages.index == _current_device() and len(ts) == 2 and ts[0] == ks[0] and table.dtype is _I32
          and table.is_contiguous() and table.get_device() == pages.index and ks[1] <= ts[1] * pages.page_tokens
          and (lens is None or (lens.dtype is _I32 and lens.shape == ks[:1] and lens.is_contiguous() and lens.get_device() == pages.index)))
    if not ok:
        _check_load(pages, table, lens, k_out, v_out)
    a = _LOAD.pack(pages.packed, table.data_ptr(), 0 if lens is None else lens.data_ptr(), k_out.data_ptr(), *kst[:3],
                   v_out.data_ptr(), *vst[:3], ks[0], ks[1], ts[1], BF16 if kind is _B16 else E5M2)
    if _fn_load is None:
        library()
    status = _fn_load(a, _stream_of(stream))
    if status:
        _check(status, "splitzip_pages_load")


def _check_load(pages, table, lens, k_out, v_out):
    for t, what in ((k_out, "k_out"), (v_out, "v_out")):
        if t.dtype != _B16 and not (t.dtype == _F8 and pages.format == E5M2):
            _bad(f"{what} is {t.dtype}: BF16, or E5M2 from pages of E5M2")
    if k_out.dtype != v_out.dtype or k_out.dim() != 4:
        _bad("k_out and v_out are [batch, tokens, kv_heads, head_dim] of one type")
    shape = (*k_out.shape[:2], pages.kv_heads, pages.head_dim)
    _check_view(k_out, shape, "k_out")
    _check_view(v_out, shape, "v_out")
    _check_table(table, lens, shape[0], shape[1], pages)
    _check_device(pages, k_out, v_out, table, lens)
    _bad("these arguments are not accepted")


def _check_table(table, lens, batch, tokens, pages):
    if table.dim() != 2:
        _bad("the table is [batch, pages of a sequence]")
    _check_array(table, _I32, (batch, table.shape[1]), "table")
    _check_array(lens, _I32, (batch,), "lens")
    if tokens > table.shape[1] * pages.page_tokens:
        _bad(f"{tokens} tokens do not fit {table.shape[1]} pages of {pages.page_tokens}")


# -------------------------------------------------------------- attention

def splitzip_paged_attention_workspace_bytes(q: torch.Tensor, pages: Pages, table: torch.Tensor, max_q_tokens: int,
                                             kv_tokens: int | None = None, window: int = 0, sinks: int = 0) -> int:
    """Workspace bytes of splitzip_paged_attention at these sizes (0: refused)."""
    if q.dim() != 3 or table.dim() != 2 or window < 0 or sinks < 0 or max_q_tokens < 0 or (kv_tokens or 0) < 0:
        return 0
    a = _ATTENTION.pack(0, 0, 0, 0, 0, 0, 0, 0, pages.packed, 0, 0, 0, 0, table.shape[0], q.shape[0], min(max_q_tokens, _MOST),
                        *_kv_tokens(kv_tokens, table, pages), q.shape[1], min(window, _MOST), min(sinks, _MOST), 1.0)
    return int(library().splitzip_paged_attention_workspace_bytes(a))


def alloc_paged_attention_workspace(q: torch.Tensor, pages: Pages, table: torch.Tensor, max_q_tokens: int,
                                    kv_tokens: int | None = None, window: int = 0, sinks: int = 0) -> torch.Tensor:
    """Zero-filled workspace for these sizes (zeroed once; reusable after).  Others, smaller ones too, may need more."""
    nbytes = splitzip_paged_attention_workspace_bytes(q, pages, table, max_q_tokens, kv_tokens, window, sinks)
    if not nbytes:
        _bad("no attention for these sizes")
    return torch.zeros(nbytes, dtype=torch.uint8, device=q.device)


def _kv_tokens(kv_tokens, table, pages):
    width = table.shape[1]
    return (min(width * pages.page_tokens, _MOST_TOKENS) if kv_tokens is None else min(kv_tokens, _MOST)), width


def splitzip_paged_attention(q: torch.Tensor, pages: Pages, table: torch.Tensor, q_start: torch.Tensor, lens: torch.Tensor,
                             out: torch.Tensor, workspace: torch.Tensor, max_q_tokens: int, kv_tokens: int | None = None,
                             lse: torch.Tensor | None = None, window: int = 0, sinks: int = 0, scale: float | None = None,
                             stream=None):
    """out = attention of the new tokens q [tokens, q_heads, head_dim] of a batch, packed, sequence b's being rows
    q_start[b] .. q_start[b + 1] - 1 (int32 [batch + 1]) and the last of its lens[b] (int32 [batch]) tokens, over
    the pages that table (int32 [batch, width]) names; asynchronous.  max_q_tokens: the most new tokens of a
    sequence; kv_tokens: the longest sequence (None: what the table holds, 2^31 - 256 at most).  lse: float32
    [q_heads, tokens] or None.  scale: None for head_dim ** -0.5.  Rows that are no sequence's stay as they were.
    ``serving.splitzip_attention_status`` reports on the workspace."""
    qs, ts = q.shape, table.shape
    qst, ost = q.stride(), out.stride()
    ok = (len(qs) == 3 and qs[2] == pages.head_dim and out.shape == qs and q.dtype is _B16 and out.dtype is _B16
          and qst[2] == 1 and ost[2] == 1 and q.get_device() == out.get_device() == pages.index == _current_device()
          and window >= 0 and sinks >= 0
          and len(ts) == 2 and table.dtype is _I32 and table.is_contiguous() and table.get_device() == pages.index
          and lens.dtype is _I32 and lens.shape == ts[:1] and lens.is_contiguous() and lens.get_device() == pages.index
          and q_start.dtype is _I32 and q_start.shape == (ts[0] + 1,) and q_start.is_contiguous() and q_start.get_device() == pages.index
          and workspace.dtype is _U8 and workspace.is_contiguous() and workspace.get_device() == pages.index
          and 0 < max_q_tokens <= qs[0] and (kv_tokens is None or 0 < kv_tokens <= ts[1] * pages.page_tokens)
          and (lse is None or (lse.dtype is _F32 and lse.shape == (qs[1], qs[0]) and lse.is_contiguous() and lse.get_device() == pages.index)))
    if not ok:
        _check_attention(q, pages, table, q_start, lens, out, workspace, max_q_tokens, kv_tokens, lse, window, sinks)
    if kv_tokens is None:
        kv_tokens = min(ts[1] * pages.page_tokens, _MOST_TOKENS)
    a = _ATTENTION.pack(q.data_ptr(), 0, qst[0], qst[1], out.data_ptr(), 0, ost[0], ost[1], pages.packed,
                        0 if lse is None else lse.data_ptr(), table.data_ptr(), q_start.data_ptr(), lens.data_ptr(),
                        ts[0], qs[0], max_q_tokens, kv_tokens if kv_tokens < _MOST else _MOST, ts[1], qs[1], window if window < _MOST else _MOST,
                        sinks if sinks < _MOST else _MOST, pages.head_dim ** -0.5 if scale is None else scale)
    if _fn_attention is None:
        library()
    status = _fn_attention(a, workspace.data_ptr(), workspace.numel(), _stream_of(stream))
    if status:
        _check(status, "splitzip_paged_attention")


def _check_attention(q, pages, table, q_start, lens, out, workspace, max_q_tokens, kv_tokens, lse, window, sinks):
    _bf16(q, "q")
    _bf16(out, "out")
    if q.dim() != 3:
        _bad("q is [tokens, q_heads, head_dim]")
    shape = (*q.shape[:2], pages.head_dim)
    _check_view(q, shape, "q")
    _check_view(out, shape, "out")
    if window < 0 or sinks < 0:
        _bad("window and sinks are not negative")
    batch = table.shape[0] if table.dim() == 2 else 0
    if lens is None or q_start is None:
        _bad("lens and q_start are needed")
    _check_table(table, lens, batch, kv_tokens or 0, pages)
    _check_array(q_start, _I32, (batch + 1,), "q_start")
    _check_array(workspace, _U8, None, "workspace")
    _check_array(lse, _F32, (shape[1], shape[0]), "lse")
    if not 0 < max_q_tokens <= shape[0]:
        _bad(f"max_q_tokens is {max_q_tokens}, of {shape[0]} tokens")
    if kv_tokens is not None and kv_tokens <= 0:
        _bad(f"kv_tokens is {kv_tokens}")
    _check_device(pages, q, out, table, q_start, lens, workspace, lse)
    _bad("these arguments are not accepted")
