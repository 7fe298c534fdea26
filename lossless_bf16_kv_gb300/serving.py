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
                ("rot_dim", _u32), ("cache_format", _u32), ("interleaved", _u32), ("eps", _f32)]


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


# The structures above as packed bytes (native layout, as the C compiler lays
# them out): a call packs its arguments in one step, which costs a fraction of
# filling a ctypes structure field by field.
_VIEW = "P3q"
_NORM_ROPE = struct.Struct("@" + 3 * _VIEW + "5P" + 3 * _VIEW + "2Q7If")
_ATTENTION = struct.Struct("@" + 4 * _VIEW + "2P9If")
_EVICT = struct.Struct("@" + 4 * _VIEW + "5P8I")
_NO_VIEW = (0, 0, 0, 0)

_lib = None


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
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
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


def _view4(t: torch.Tensor, shape, what: str) -> tuple:
    """(pointer, stride_b, stride_t, stride_h) of a [batch, tokens, heads, dim] view."""
    if t.shape != shape:
        _bad(f"{what} has shape {tuple(t.shape)}, {tuple(shape)} needed")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    sb, st, sh, one = t.stride()
    if one != 1:
        _bad(f"{what}: the values of a row must be contiguous")
    return t.data_ptr(), sb, st, sh


def _view3(t: torch.Tensor, shape, what: str) -> tuple:
    """(pointer, 0, stride_t, stride_h) of a [tokens, heads, dim] view."""
    if t.shape != shape:
        _bad(f"{what} has shape {tuple(t.shape)}, {tuple(shape)} needed")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    st, sh, one = t.stride()
    if one != 1:
        _bad(f"{what}: the values of a row must be contiguous")
    return t.data_ptr(), 0, st, sh


def _array(t: torch.Tensor | None, dtype, shape: tuple | None, what: str) -> int:
    """Pointer of a contiguous array of this type and shape, or 0 for None."""
    if t is None:
        return 0
    if t.dtype != dtype:
        _bad(f"{what} is {t.dtype}, {dtype} needed")
    if shape is not None and t.shape != shape:
        _bad(f"{what} has shape {tuple(t.shape)}, {shape} needed")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor")
    return t.data_ptr()


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
    """(rows, pointer, stride_t, stride_h) of a cache addressed by row: [rows,
    heads, dim], or [batch, tokens, heads, dim] whose batch stride is a whole
    number of token strides (row = b * stride_b // stride_t + token)."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    shape, st = t.shape, t.stride()
    if st[-1] != 1:
        _bad(f"{what}: the values of a row must be contiguous")
    if len(shape) == 3:
        return shape[0], t.data_ptr(), st[0], st[1]
    if len(shape) != 4:
        _bad(f"{what} is [rows, heads, dim] or [batch, tokens, heads, dim]")
    if shape[0] > 1 and (st[1] == 0 or st[0] % st[1]):
        _bad(f"{what}: the batch stride must be a multiple of the token stride")
    rows = (shape[0] - 1) * (st[0] // st[1]) + shape[1] if shape[0] > 1 else shape[0] * shape[1]
    return rows, t.data_ptr(), st[1], st[2]


def splitzip_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_weight, k_weight, positions, table,
                          slots: torch.Tensor, q_out: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          eps: float = 1e-6, interleaved: bool = False, stream=None):
    """Norm and rotate q [n, q_heads, dim] into q_out and k [n, kv_heads, dim]
    into k_cache[slots], store v into v_cache[slots]; asynchronous.

    q_weight, k_weight: BF16 [dim] or None.  table: float32 [positions, rot_dim]
    (cosines, then sines) or None for no rotation; positions int32 [n].
    slots: int64 [n]; a cache [batch, tokens, heads, dim] is addressed by
    b * stride_b // stride_t + token.  q_out may be q."""
    n, hq, dim = q.shape
    hk = k.shape[1]
    for t, what in ((q, "q"), (k, "k"), (v, "v"), (q_out, "q_out")):
        _bf16(t, what)
    fmt = _format(k_cache, v_cache)
    krows, kp, kst, ksh = _cache_rows(k_cache, "k_cache")
    vrows, vp, vst, vsh = _cache_rows(v_cache, "v_cache")
    if k_cache.shape[-2:] != (hk, dim) or v_cache.shape[-2:] != (hk, dim):
        _bad("the caches' heads and dims must be those of k")
    rot = 0
    if table is not None:
        if table.dim() != 2:
            _bad("table is [positions, rot_dim]")
        rot = table.shape[1]
        if positions is None:
            _bad("a rotation needs positions")
    kshape = (n, hk, dim)
    a = _NORM_ROPE.pack(*_view3(q, q.shape, "q"), *_view3(k, kshape, "k"), *_view3(v, kshape, "v"),
                        _array(q_weight, torch.bfloat16, (dim,), "q_weight"),
                        _array(k_weight, torch.bfloat16, (dim,), "k_weight"),
                        _array(positions, torch.int32, (n,), "positions"),
                        _array(table, torch.float32, None, "table"), _array(slots, torch.int64, (n,), "slots"),
                        *_view3(q_out, q.shape, "q_out"), kp, 0, kst, ksh, vp, 0, vst, vsh,
                        table.shape[0] if rot else 0, min(krows, vrows), n, hq, hk, dim, rot, fmt, bool(interleaved), eps)
    _check((_lib or library()).splitzip_qk_norm_rope(a, _stream_of(stream)), "splitzip_qk_norm_rope")


# ------------------------------------------------------------- attention

def _sizes(q_shape, k_shape, fmt: int, window: int, sinks: int):
    if len(q_shape) != 4 or len(k_shape) != 4:
        _bad("q and the caches are [batch, tokens, heads, dim]")
    if window < 0 or sinks < 0:
        _bad("window and sinks are not negative")
    return (q_shape[0], q_shape[1], k_shape[1], q_shape[2], k_shape[2], q_shape[3],
            min(window, 0x80000000), min(sinks, 0x80000000), fmt)


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


def splitzip_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, out: torch.Tensor,
                       workspace: torch.Tensor, lens: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       window: int = 0, sinks: int = 0, scale: float | None = None, stream=None):
    """out = attention of q [batch, q_tokens, q_heads, dim] over the caches
    [batch, kv_tokens, kv_heads, dim]; asynchronous.  The queries are the last
    q_tokens of lens[b] (int32; None: kv_tokens) tokens.  lse: float32 [batch,
    q_heads, q_tokens] or None.  scale: None for dim ** -0.5."""
    qs, ks = q.shape, k_cache.shape
    fmt = _format(k_cache, v_cache)
    sizes = _sizes(qs, ks, fmt, window, sinks)
    b, tq, tk, hq, hk, dim = sizes[:6]
    _bf16(q, "q")
    _bf16(out, "out")
    if ks[0] != b or ks[3] != dim:
        _bad("q's batch and dims must be the caches'")
    a = _ATTENTION.pack(*_view4(q, qs, "q"), *_view4(k_cache, ks, "k_cache"), *_view4(v_cache, ks, "v_cache"),
                        *_view4(out, qs, "out"), _array(lse, torch.float32, (b, hq, tq), "lse"),
                        _array(lens, torch.int32, (b,), "lens"), *sizes, dim ** -0.5 if scale is None else scale)
    _check((_lib or library()).splitzip_attention(a, _array(workspace, torch.uint8, None, "workspace"),
                                                  workspace.numel(), _stream_of(stream)), "splitzip_attention")


def splitzip_attention_status(workspace: torch.Tensor, stream=None) -> int:
    """Status of the attention calls on this workspace since the last report
    (OK or ERR_TIMEOUT); synchronises the stream."""
    return int(library().splitzip_attention_status(_array(workspace, torch.uint8, None, "workspace"), _stream_of(stream)))


def splitzip_attention_weights(q: torch.Tensor, k_cache: torch.Tensor, lse: torch.Tensor, weights_out: torch.Tensor,
                               lens: torch.Tensor | None = None, weights_in: torch.Tensor | None = None,
                               window: int = 0, sinks: int = 0, scale: float | None = None, stream=None):
    """weights_out [batch, kv_heads, kv_tokens] = weights_in (or 0) + the softmax
    weight each slot gets from q's rows, whose lse splitzip_attention returned;
    asynchronous.  To weigh the tokens by the last queries only, pass those
    queries and their lse."""
    qs, ks = q.shape, k_cache.shape
    sizes = _sizes(qs, ks, _format(k_cache), window, sinks)
    b, tq, tk, hq, hk, dim = sizes[:6]
    _bf16(q, "q")
    if ks[0] != b or ks[3] != dim:
        _bad("q's batch and dims must be the cache's")
    if lse is None or weights_out is None:
        _bad("lse and weights_out are needed")
    a = _ATTENTION.pack(*_view4(q, qs, "q"), *_view4(k_cache, ks, "k_cache"), *_NO_VIEW, *_NO_VIEW,
                        _array(lse, torch.float32, (b, hq, tq), "lse"), _array(lens, torch.int32, (b,), "lens"),
                        *sizes, dim ** -0.5 if scale is None else scale)
    _check((_lib or library()).splitzip_attention_weights(
        a, _array(weights_in, torch.float32, (b, hk, tk), "weights_in"),
        _array(weights_out, torch.float32, (b, hk, tk), "weights_out"), _stream_of(stream)),
        "splitzip_attention_weights")


# -------------------------------------------------------------- eviction

def splitzip_evict(k_cache: torch.Tensor, v_cache: torch.Tensor, weights: torch.Tensor, k_out: torch.Tensor,
                   v_out: torch.Tensor, index: torch.Tensor, lens: torch.Tensor | None = None,
                   weights_out: torch.Tensor | None = None, lens_out: torch.Tensor | None = None,
                   keep_first: int = 0, keep_last: int = 0, stream=None):
    """Keep, per sequence and head, the first keep_first, the last keep_last and
    the most attended slots, k_out.shape[1] in all; index [batch, kv_heads,
    budget] int32 receives the old slots, in order; asynchronous."""
    ks, os = k_cache.shape, k_out.shape
    fmt = _format(k_cache, v_cache)
    if _format(k_out, v_out) != fmt:
        _bad("the outputs must have the cache's type")
    if len(ks) != 4 or len(os) != 4 or (os[0], *os[2:]) != (ks[0], *ks[2:]):
        _bad("the outputs must be [batch, budget, kv_heads, dim] of the cache")
    if keep_first < 0 or keep_last < 0:
        _bad("keep_first and keep_last are not negative")
    b, t, h, dim = ks
    budget = os[1]
    a = _EVICT.pack(*_view4(k_cache, ks, "k_cache"), *_view4(v_cache, ks, "v_cache"), *_view4(k_out, os, "k_out"),
                    *_view4(v_out, os, "v_out"), _array(weights, torch.float32, (b, h, t), "weights"),
                    _array(lens, torch.int32, (b,), "lens"), _array(index, torch.int32, (b, h, budget), "index"),
                    _array(weights_out, torch.float32, (b, h, budget), "weights_out"),
                    _array(lens_out, torch.int32, (b,), "lens_out"), b, t, h, dim, budget, keep_first, keep_last, fmt)
    _check((_lib or library()).splitzip_evict(a, _stream_of(stream)), "splitzip_evict")
