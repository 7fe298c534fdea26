"""Thin Python binding of include/splitzip_serving.h: the operators around a KV
cache (norm and rotation into it, attention over it, the attention weight of
its tokens, eviction from it).

Argument marshalling only, as in ``splitzip``: PyTorch supplies device memory
and streams, everything runs in the library's CUDA kernels on the current
stream (or ``stream``), nothing is allocated or synchronised.  The C ABI takes
plain pointers, so shapes, types and the extent of every buffer are checked
here (``SplitZipError`` with ``ERR_INVALID_ARG``); strides and alignment are
checked by the library.

Caches are views [batch, tokens, kv_heads, head_dim] of BF16 or FP8 E5M2, for
instance ``kv[:, 0]`` and ``kv[:, 1]`` of a tensor [layers, 2, tokens,
kv_heads, head_dim].
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import splitzip as _sz
from .splitzip import ERR_INVALID_ARG, SplitZipError

BF16, E5M2 = 0, 1
_FORMAT = {torch.bfloat16: BF16, torch.float8_e5m2: E5M2}
_u32, _u64, _i64, _f32, _vp = (ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int64, ctypes.c_float,
                               ctypes.c_void_p)


class View(ctypes.Structure):
    _fields_ = [("data", _vp), ("stride_b", _i64), ("stride_t", _i64), ("stride_h", _i64)]


class NormRopeArgs(ctypes.Structure):
    _fields_ = [("q", View), ("k", View), ("v", View), ("q_weight", _vp), ("k_weight", _vp),
                ("positions", _vp), ("table", _vp), ("slots", _vp),
                ("q_out", View), ("k_cache", View), ("v_cache", View),
                ("table_rows", _u64), ("cache_rows", _u64),
                ("n", _u32), ("q_heads", _u32), ("kv_heads", _u32), ("head_dim", _u32),
                ("rot_dim", _u32), ("cache_format", _u32), ("interleaved", _u32), ("eps", _f32),
                ("cache_step", _u32), ("cache_tokens", _u32)]


class AttentionArgs(ctypes.Structure):
    _fields_ = [("q", View), ("k", View), ("v", View), ("out", View), ("lse", _vp), ("lens", _vp),
                ("batch", _u32), ("q_tokens", _u32), ("kv_tokens", _u32), ("q_heads", _u32),
                ("kv_heads", _u32), ("head_dim", _u32), ("window", _u32), ("sinks", _u32),
                ("cache_format", _u32), ("scale", _f32)]


class EvictArgs(ctypes.Structure):
    _fields_ = [("k", View), ("v", View), ("k_out", View), ("v_out", View),
                ("weights", _vp), ("lens", _vp), ("index", _vp), ("weights_out", _vp), ("lens_out", _vp),
                ("batch", _u32), ("kv_tokens", _u32), ("kv_heads", _u32), ("head_dim", _u32),
                ("budget", _u32), ("keep_first", _u32), ("keep_last", _u32), ("cache_format", _u32)]


class WaitTestOpts(ctypes.Structure):
    """Test controls (include/splitzip_serving_testing.h)."""
    _fields_ = [("wait_ms", _u32), ("cta", _u32), ("tile", _u32)]


# The structures above as packed bytes (native layout, as the C compiler lays
# them out): a call packs its arguments in one step, which costs a fraction of
# filling a ctypes structure field by field.
_VIEW = "P3q"
_NORM_ROPE = struct.Struct("@" + 3 * _VIEW + "5P" + 3 * _VIEW + "2Q7If2I")
_ATTENTION = struct.Struct("@" + 4 * _VIEW + "2P9If")
_EVICT = struct.Struct("@" + 4 * _VIEW + "5P8I")
_NO_VIEW = (0, 0, 0, 0)

_lib = None
_fn_norm_rope = _fn_attention = _fn_weights = _fn_evict = None
_B16, _F8, _F32, _I32, _I64, _U8 = (torch.bfloat16, torch.float8_e5m2, torch.float32, torch.int32, torch.int64,
                                    torch.uint8)


def library() -> ctypes.CDLL:
    """libsplitzip.so with the signatures of splitzip_serving.h (raises if it
    has not been built)."""
    global _lib
    if _lib is None:
        lib = _sz.library()
        sig = {
            "splitzip_qk_norm_rope": (ctypes.c_int, [_vp, _vp]),
            "splitzip_attention_workspace_bytes": (ctypes.c_size_t, [_vp]),
            "splitzip_attention": (ctypes.c_int, [_vp, _vp, ctypes.c_size_t, _vp]),
            "splitzip_attention_status": (ctypes.c_int, [_vp, _vp]),
            "splitzip_attention_weights": (ctypes.c_int, [_vp, _vp, _vp, _vp]),
            "splitzip_evict": (ctypes.c_int, [_vp, _vp]),
            "splitzip_attention_test": (ctypes.c_int, [_vp, _vp, ctypes.c_size_t, _vp, _vp]),
            "splitzip_attention_weights_test": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
        global _fn_norm_rope, _fn_attention, _fn_weights, _fn_evict
        _fn_norm_rope, _fn_attention = lib.splitzip_qk_norm_rope, lib.splitzip_attention
        _fn_weights, _fn_evict = lib.splitzip_attention_weights, lib.splitzip_evict
    return _lib


def _bad(what: str):
    raise SplitZipError(ERR_INVALID_ARG, what)


def _check(status: int, what: str):
    if status:
        raise SplitZipError(status, what)


_current_device = torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without a Stream object


def _stream_of(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(_current_device())
    return torch.cuda.current_stream().cuda_stream


# A call on small tensors costs less than looking at its arguments, so each
# function checks them in one expression; only where that fails are they gone
# through one by one, to say which is wrong.

def _check_view(t: torch.Tensor, shape, what: str):
    if tuple(t.shape) != tuple(shape):
        _bad(f"{what} has shape {tuple(t.shape)}, {tuple(shape)} needed")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.stride()[-1] != 1:
        _bad(f"{what}: the values of a row must be contiguous")


def _check_array(t: torch.Tensor | None, dtype, shape: tuple | None, what: str):
    """A contiguous array of this type and shape, or None."""
    if t is None:
        return
    if t.dtype != dtype:
        _bad(f"{what} is {t.dtype}, {dtype} needed")
    if shape is not None and tuple(t.shape) != tuple(shape):
        _bad(f"{what} has shape {tuple(t.shape)}, {tuple(shape)} needed")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor")


def _bf16(t: torch.Tensor, what: str):
    if t.dtype != torch.bfloat16:
        _bad(f"{what} is {t.dtype}, torch.bfloat16 needed")


def _format(k: torch.Tensor, v: torch.Tensor | None = None) -> int:
    fmt = _FORMAT.get(k.dtype)
    if fmt is None:
        _bad(f"a cache is BF16 or E5M2, not {k.dtype}")
    if v is not None and v.dtype != k.dtype:
        _bad(f"keys are {k.dtype}, values {v.dtype}")
    return fmt


# --------------------------------------------------- norm, rotation, cache

def _cache_rows(t: torch.Tensor, what: str) -> tuple:
    """(rows, stride_t, stride_h, step) of a cache addressed by row: [rows, heads,
    dim], or [batch, tokens, heads, dim] whose batch stride is a whole number of
    token strides (row = b * stride_b // stride_t + token).  step is that number
    where it leaves gaps between the sequences, else 0."""
    shape, st = t.shape, t.stride()
    if st[-1] != 1:
        _bad(f"{what}: the values of a row must be contiguous")
    if len(shape) == 3:
        return shape[0], st[0], st[1], 0
    if len(shape) != 4:
        _bad(f"{what} is [rows, heads, dim] or [batch, tokens, heads, dim]")
    if shape[0] > 1 and (st[1] == 0 or st[0] % st[1]):
        _bad(f"{what}: the batch stride must be a multiple of the token stride")
    if shape[0] <= 1:
        return shape[0] * shape[1], st[1], st[2], 0
    step = st[0] // st[1]
    return (shape[0] - 1) * step + shape[1], st[1], st[2], step if step > shape[1] else 0


def _check_same_rows(k_cache: torch.Tensor, v_cache: torch.Tensor, kstep: int, vstep: int):
    """One slot addresses both caches: it must be the same sequence's same token in both."""
    ks, vs, kst, vst = k_cache.shape, v_cache.shape, k_cache.stride(), v_cache.stride()
    if len(ks) == 4 and len(vs) == 4 and ks[0] > 1 and vs[0] > 1:
        if ks != vs:
            _bad(f"batched caches must have one shape, not {tuple(ks)} and {tuple(vs)}")
        if kst[0] * vst[1] != vst[0] * kst[1]:
            _bad("the caches' sequences must be the same number of tokens apart")
    elif kstep or vstep:
        _bad("a cache with gaps between its sequences needs the other one like it")


def _check_norm_rope(q, k, v, q_weight, k_weight, positions, table, slots, q_out, k_cache, v_cache):
    for t, what in ((q, "q"), (k, "k"), (v, "v"), (q_out, "q_out")):
        _bf16(t, what)
        if t.dim() != 3:
            _bad(f"{what} is [tokens, heads, dim]")
    _format(k_cache, v_cache)
    n, _, dim = q.shape
    hk = k.shape[1]
    _check_view(q, q.shape, "q")
    _check_view(k, (n, hk, dim), "k")
    _check_view(v, (n, hk, dim), "v")
    _check_view(q_out, q.shape, "q_out")
    for t, what in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not t.is_cuda:
            raise ValueError(f"{what} must be a CUDA tensor")
        if tuple(t.shape[-2:]) != (hk, dim):
            _bad("the caches' heads and dims must be those of k")
    _check_array(q_weight, _B16, (dim,), "q_weight")
    _check_array(k_weight, _B16, (dim,), "k_weight")
    if slots is None:
        _bad("slots are needed")
    _check_array(slots, _I64, (n,), "slots")
    _check_array(positions, _I32, (n,), "positions")
    _check_array(table, _F32, None, "table")
    if table is not None and (table.dim() != 2 or positions is None):
        _bad("a rotation needs a table [positions, rot_dim] and positions")
    _bad("these arguments are not accepted")


def splitzip_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_weight, k_weight, positions, table,
                          slots: torch.Tensor, q_out: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          eps: float = 1e-6, interleaved: bool = False, stream=None):
    """Norm and rotate q [n, q_heads, dim] into q_out and k [n, kv_heads, dim]
    into k_cache[slots], store v into v_cache[slots]; asynchronous.

    q_weight, k_weight: BF16 [dim] or None.  table: float32 [positions, rot_dim]
    (cosines, then sines) or None for no rotation; positions int32 [n].
    slots: int64 [n]; a cache [batch, tokens, heads, dim] is addressed by
    b * stride_b // stride_t + token; a slot that is no row of the cache is
    dropped, one between two sequences too.  q_out may be q."""
    qs, ks, kind = q.shape, k.shape, k_cache.dtype
    qst, kst, vst, ost = q.stride(), k.stride(), v.stride(), q_out.stride()
    cs, rot = k_cache.shape, 0
    ok = (len(qs) == 3 and len(ks) == 3 and qs[0] == ks[0] and qs[2] == ks[2] and v.shape == ks and q_out.shape == qs
          and q.dtype is _B16 and k.dtype is _B16 and v.dtype is _B16 and q_out.dtype is _B16
          and (kind is _B16 or kind is _F8) and v_cache.dtype is kind
          and qst[2] == 1 and kst[2] == 1 and vst[2] == 1 and ost[2] == 1
          and cs[-2:] == ks[1:] and v_cache.shape[-2:] == ks[1:]
          and slots is not None and slots.dtype is _I64 and slots.shape == qs[:1] and slots.is_contiguous()
          and q.is_cuda and k.is_cuda and v.is_cuda and q_out.is_cuda and k_cache.is_cuda and v_cache.is_cuda
          and slots.is_cuda)
    for w in (q_weight, k_weight):
        ok = ok and (w is None or (w.dtype is _B16 and w.shape == qs[2:] and w.is_contiguous() and w.is_cuda))
    if ok and table is not None:
        ts = table.shape
        ok = (len(ts) == 2 and table.dtype is _F32 and table.is_contiguous() and table.is_cuda
              and positions is not None and positions.dtype is _I32 and positions.shape == qs[:1]
              and positions.is_contiguous() and positions.is_cuda)
        rot = ts[1] if ok else 0
    if not ok:
        _check_norm_rope(q, k, v, q_weight, k_weight, positions, table, slots, q_out, k_cache, v_cache)
    krows, kct, kch, step = _cache_rows(k_cache, "k_cache")
    vrows, vct, vch, vstep = _cache_rows(v_cache, "v_cache")
    if len(cs) == 4 or len(v_cache.shape) == 4:
        _check_same_rows(k_cache, v_cache, step, vstep)
    a = _NORM_ROPE.pack(q.data_ptr(), 0, qst[0], qst[1], k.data_ptr(), 0, kst[0], kst[1], v.data_ptr(), 0, vst[0], vst[1],
                        0 if q_weight is None else q_weight.data_ptr(), 0 if k_weight is None else k_weight.data_ptr(),
                        positions.data_ptr() if rot else 0, table.data_ptr() if rot else 0, slots.data_ptr(),
                        q_out.data_ptr(), 0, ost[0], ost[1], k_cache.data_ptr(), 0, kct, kch, v_cache.data_ptr(), 0, vct, vch,
                        ts[0] if rot else 0, krows if krows < vrows else vrows, *qs[:2], *ks[1:], rot, _FORMAT[kind],
                        1 if interleaved else 0, eps, step, cs[1] if step else 0)
    if _fn_norm_rope is None:
        library()
    status = _fn_norm_rope(a, _stream_of(stream))
    if status:
        _check(status, "splitzip_qk_norm_rope")


# ------------------------------------------------------------- attention

def _sizes(q_shape, k_shape, fmt: int, window: int, sinks: int):
    if len(q_shape) != 4 or len(k_shape) != 4:
        _bad("q and the caches are [batch, tokens, heads, dim]")
    if window < 0 or sinks < 0:
        _bad("window and sinks are not negative")
    return (q_shape[0], q_shape[1], k_shape[1], q_shape[2], k_shape[2], q_shape[3],
            min(window, _MOST), min(sinks, _MOST), fmt)


def splitzip_attention_workspace_bytes(q: torch.Tensor, k_cache: torch.Tensor, window: int = 0, sinks: int = 0) -> int:
    """Workspace bytes of splitzip_attention at these sizes (0: refused)."""
    a = _ATTENTION.pack(*_NO_VIEW, *_NO_VIEW, *_NO_VIEW, *_NO_VIEW, 0, 0,
                        *_sizes(q.shape, k_cache.shape, _format(k_cache), window, sinks), 1.0)
    return int(library().splitzip_attention_workspace_bytes(a))


def alloc_attention_workspace(q: torch.Tensor, k_cache: torch.Tensor, window: int = 0, sinks: int = 0) -> torch.Tensor:
    """Zero-filled workspace for these sizes (zeroed once; reusable after)."""
    nbytes = splitzip_attention_workspace_bytes(q, k_cache, window, sinks)
    if not nbytes:
        _bad("no attention for these sizes")
    return torch.zeros(nbytes, dtype=torch.uint8, device=q.device)


_MOST = 0x80000000   # a longer window is unlimited too


def _check_attention(q, k_cache, v_cache, out, workspace, lens, lse, window, sinks):
    fmt = _format(k_cache, v_cache)
    b, tq, _, hq, _, dim = _sizes(q.shape, k_cache.shape, fmt, window, sinks)[:6]
    _bf16(q, "q")
    _bf16(out, "out")
    if k_cache.shape[0] != b or k_cache.shape[3] != dim:
        _bad("q's batch and dims must be the caches'")
    for t, like, what in ((q, q, "q"), (k_cache, k_cache, "k_cache"), (v_cache, k_cache, "v_cache"), (out, q, "out")):
        _check_view(t, like.shape, what)
    _check_array(workspace, _U8, None, "workspace")
    _check_array(lens, _I32, (b,), "lens")
    _check_array(lse, _F32, (b, hq, tq), "lse")
    _bad("these arguments are not accepted")


def _check_weights(q, k_cache, lse, weights_out, lens, weights_in, window, sinks):
    b, tq, tk, hq, hk, dim = _sizes(q.shape, k_cache.shape, _format(k_cache), window, sinks)[:6]
    _bf16(q, "q")
    if k_cache.shape[0] != b or k_cache.shape[3] != dim:
        _bad("q's batch and dims must be the cache's")
    if lse is None or weights_out is None:
        _bad("lse and weights_out are needed")
    _check_view(q, q.shape, "q")
    _check_view(k_cache, k_cache.shape, "k_cache")
    _check_array(lse, _F32, (b, hq, tq), "lse")
    _check_array(lens, _I32, (b,), "lens")
    _check_array(weights_in, _F32, (b, hk, tk), "weights_in")
    _check_array(weights_out, _F32, (b, hk, tk), "weights_out")
    _bad("these arguments are not accepted")


def splitzip_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, out: torch.Tensor,
                       workspace: torch.Tensor, lens: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       window: int = 0, sinks: int = 0, scale: float | None = None, stream=None):
    """out = attention of q [batch, q_tokens, q_heads, dim] over the caches
    [batch, kv_tokens, kv_heads, dim]; asynchronous.  The queries are the last
    q_tokens of lens[b] (int32; None: kv_tokens) tokens.  lse: float32 [batch,
    q_heads, q_tokens] or None.  scale: None for dim ** -0.5."""
    qs, ks, kind = q.shape, k_cache.shape, k_cache.dtype
    qst, kst, vst, ost = q.stride(), k_cache.stride(), v_cache.stride(), out.stride()
    ok = (len(qs) == 4 and len(ks) == 4 and qs[0] == ks[0] and qs[3] == ks[3] and v_cache.shape == ks and out.shape == qs
          and q.dtype is _B16 and out.dtype is _B16 and (kind is _B16 or kind is _F8) and v_cache.dtype is kind
          and qst[3] == 1 and kst[3] == 1 and vst[3] == 1 and ost[3] == 1 and window >= 0 and sinks >= 0
          and q.is_cuda and k_cache.is_cuda and v_cache.is_cuda and out.is_cuda
          and workspace.dtype is _U8 and workspace.is_contiguous() and workspace.is_cuda
          and (lens is None or (lens.dtype is _I32 and lens.shape == qs[:1] and lens.is_contiguous() and lens.is_cuda))
          and (lse is None or (lse.dtype is _F32 and lse.shape == (qs[0], qs[2], qs[1]) and lse.is_contiguous()
                               and lse.is_cuda)))
    if not ok:
        _check_attention(q, k_cache, v_cache, out, workspace, lens, lse, window, sinks)
    a = _ATTENTION.pack(q.data_ptr(), *qst[:3], k_cache.data_ptr(), *kst[:3], v_cache.data_ptr(), *vst[:3],
                        out.data_ptr(), *ost[:3], 0 if lse is None else lse.data_ptr(),
                        0 if lens is None else lens.data_ptr(), qs[0], qs[1], ks[1], qs[2], ks[2], qs[3],
                        window if window < _MOST else _MOST, sinks if sinks < _MOST else _MOST, _FORMAT[kind],
                        qs[3] ** -0.5 if scale is None else scale)
    if _fn_attention is None:
        library()
    status = _fn_attention(a, workspace.data_ptr(), workspace.numel(), _stream_of(stream))
    if status:
        _check(status, "splitzip_attention")


_HEADER = 1024   # bytes that every workspace begins with: counters, then the status in the last word


def splitzip_attention_status(workspace: torch.Tensor, stream=None) -> int:
    """Status of the attention calls on this workspace since the last report
    (OK or ERR_TIMEOUT); synchronises the stream."""
    _check_array(workspace, _U8, None, "workspace")
    if workspace.numel() < _HEADER:
        _bad(f"a workspace of {workspace.numel()} bytes is none of splitzip_attention's")
    return int(library().splitzip_attention_status(workspace.data_ptr(), _stream_of(stream)))


def splitzip_attention_weights(q: torch.Tensor, k_cache: torch.Tensor, lse: torch.Tensor, weights_out: torch.Tensor,
                               lens: torch.Tensor | None = None, weights_in: torch.Tensor | None = None,
                               window: int = 0, sinks: int = 0, scale: float | None = None, stream=None):
    """weights_out [batch, kv_heads, kv_tokens] = weights_in (or 0) + the softmax
    weight each slot gets from q's rows, whose lse splitzip_attention returned;
    asynchronous.  To weigh the tokens by the last queries only, pass those
    queries and their lse."""
    qs, ks, kind = q.shape, k_cache.shape, k_cache.dtype
    qst, kst = q.stride(), k_cache.stride()
    ok = (len(qs) == 4 and len(ks) == 4 and qs[0] == ks[0] and qs[3] == ks[3] and q.dtype is _B16
          and (kind is _B16 or kind is _F8) and qst[3] == 1 and kst[3] == 1 and window >= 0 and sinks >= 0
          and q.is_cuda and k_cache.is_cuda and lse is not None and lse.dtype is _F32
          and lse.shape == (qs[0], qs[2], qs[1]) and lse.is_contiguous() and lse.is_cuda)
    if ok:
        ws = (ks[0], ks[2], ks[1])
        ok = (weights_out is not None and weights_out.dtype is _F32 and weights_out.shape == ws
              and weights_out.is_contiguous() and weights_out.is_cuda
              and (weights_in is None or weights_in is weights_out or (
                  weights_in.dtype is _F32 and weights_in.shape == ws and weights_in.is_contiguous() and weights_in.is_cuda))
              and (lens is None or (lens.dtype is _I32 and lens.shape == qs[:1] and lens.is_contiguous() and lens.is_cuda)))
    if not ok:
        _check_weights(q, k_cache, lse, weights_out, lens, weights_in, window, sinks)
    a = _ATTENTION.pack(q.data_ptr(), *qst[:3], k_cache.data_ptr(), *kst[:3], *_NO_VIEW, *_NO_VIEW, lse.data_ptr(),
                        0 if lens is None else lens.data_ptr(), qs[0], qs[1], ks[1], qs[2], ks[2], qs[3],
                        window if window < _MOST else _MOST, sinks if sinks < _MOST else _MOST, _FORMAT[kind],
                        qs[3] ** -0.5 if scale is None else scale)
    if _fn_weights is None:
        library()
    status = _fn_weights(a, 0 if weights_in is None else weights_in.data_ptr(), weights_out.data_ptr(), _stream_of(stream))
    if status:
        _check(status, "splitzip_attention_weights")


# -------------------------------------------------------------- eviction

def splitzip_evict(k_cache: torch.Tensor, v_cache: torch.Tensor, weights: torch.Tensor, k_out: torch.Tensor,
                   v_out: torch.Tensor, index: torch.Tensor, lens: torch.Tensor | None = None,
                   weights_out: torch.Tensor | None = None, lens_out: torch.Tensor | None = None,
                   keep_first: int = 0, keep_last: int = 0, stream=None):
    """Keep, per sequence and head, the first keep_first, the last keep_last and
    the most attended slots, k_out.shape[1] in all; index [batch, kv_heads,
    budget] int32 receives the old slots, in order; asynchronous."""
    ks, os, kind = k_cache.shape, k_out.shape, k_cache.dtype
    kst, vst, kot, vot = k_cache.stride(), v_cache.stride(), k_out.stride(), v_out.stride()
    ok = (len(ks) == 4 and len(os) == 4 and os[0] == ks[0] and os[2:] == ks[2:] and v_cache.shape == ks and v_out.shape == os
          and (kind is _B16 or kind is _F8) and v_cache.dtype is kind and k_out.dtype is kind and v_out.dtype is kind
          and kst[3] == 1 and vst[3] == 1 and kot[3] == 1 and vot[3] == 1 and keep_first >= 0 and keep_last >= 0
          and k_cache.is_cuda and v_cache.is_cuda and k_out.is_cuda and v_out.is_cuda)
    if ok:
        b, t, h, dim = ks
        budget = os[1]
        kept = (b, h, budget)
        ok = (weights.dtype is _F32 and weights.shape == (b, h, t) and weights.is_contiguous() and weights.is_cuda
              and index.dtype is _I32 and index.shape == kept and index.is_contiguous() and index.is_cuda
              and (weights_out is None or (weights_out.dtype is _F32 and weights_out.shape == kept
                                           and weights_out.is_contiguous() and weights_out.is_cuda))
              and (lens is None or (lens.dtype is _I32 and lens.shape == ks[:1] and lens.is_contiguous() and lens.is_cuda))
              and (lens_out is None or (lens_out.dtype is _I32 and lens_out.shape == ks[:1] and lens_out.is_contiguous()
                                        and lens_out.is_cuda)))
    if not ok:
        _check_evict(k_cache, v_cache, weights, k_out, v_out, index, lens, weights_out, lens_out, keep_first, keep_last)
    a = _EVICT.pack(k_cache.data_ptr(), *kst[:3], v_cache.data_ptr(), *vst[:3], k_out.data_ptr(), *kot[:3],
                    v_out.data_ptr(), *vot[:3], weights.data_ptr(), 0 if lens is None else lens.data_ptr(), index.data_ptr(),
                    0 if weights_out is None else weights_out.data_ptr(), 0 if lens_out is None else lens_out.data_ptr(),
                    b, t, h, dim, budget, keep_first if keep_first < _MOST else _MOST,
                    keep_last if keep_last < _MOST else _MOST, _FORMAT[kind])
    if _fn_evict is None:
        library()
    status = _fn_evict(a, _stream_of(stream))
    if status:
        _check(status, "splitzip_evict")


def _check_evict(k_cache, v_cache, weights, k_out, v_out, index, lens, weights_out, lens_out, keep_first, keep_last):
    if _format(k_out, v_out) != _format(k_cache, v_cache):
        _bad("the outputs must have the cache's type")
    ks, os = tuple(k_cache.shape), tuple(k_out.shape)
    if len(ks) != 4 or len(os) != 4 or (os[0], *os[2:]) != (ks[0], *ks[2:]):
        _bad("the outputs must be [batch, budget, kv_heads, dim] of the cache")
    if keep_first < 0 or keep_last < 0:
        _bad("keep_first and keep_last are not negative")
    for x, shape, what in ((k_cache, ks, "k_cache"), (v_cache, ks, "v_cache"), (k_out, os, "k_out"), (v_out, os, "v_out")):
        _check_view(x, shape, what)
    b, t, h, _ = ks
    _check_array(weights, _F32, (b, h, t), "weights")
    _check_array(index, _I32, (b, h, os[1]), "index")
    _check_array(weights_out, _F32, (b, h, os[1]), "weights_out")
    _check_array(lens, _I32, (b,), "lens")
    _check_array(lens_out, _I32, (b,), "lens_out")
    _bad("these arguments are not accepted")
