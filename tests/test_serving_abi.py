"""include/splitzip_serving.h on the CPU: its functions are exported and bound,
the binding's structures have the C ones' layout, and every argument that the
host checks refuse is refused before anything is enqueued (no GPU is needed to
see that)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from lossless_bf16_kv_gb300 import _build, serving
from lossless_bf16_kv_gb300 import splitzip as sz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "splitzip_serving.h")
STRUCTS = {"splitzip_view": serving.View, "splitzip_norm_rope_args": serving.NormRopeArgs,
           "splitzip_attention_args": serving.AttentionArgs, "splitzip_evict_args": serving.EvictArgs}


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return serving.library()


def test_library_exports_and_binds_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(splitzip_\w+)\s*\(", text)))
    assert len(names) == 6
    for name in names:
        assert getattr(lib, name).argtypes is not None, name


def test_structures_have_the_c_layout(tmp_path):
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("%zu ", sizeof({name}));')
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu ", offsetof({name}, {f}));')
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "splitzip_serving.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", f"-I{ROOT}/include", str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for cls in STRUCTS.values():
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want
    assert [x.size for x in (serving._NORM_ROPE, serving._ATTENTION, serving._EVICT)] == \
        [ctypes.sizeof(x) for x in (serving.NormRopeArgs, serving.AttentionArgs, serving.EvictArgs)]


FAKE = 1 << 20   # aligned, never dereferenced: every call below is refused


def attention_args(**kw):
    view = (FAKE, 1 << 16, 1 << 10, 128)
    a = serving.AttentionArgs(view, view, view, view, FAKE, FAKE, 2, 3, 64, 8, 2, 128, 0, 0, 0, 1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(q_tokens=0), dict(kv_tokens=0), dict(q_heads=0), dict(kv_heads=0), dict(head_dim=96),
    dict(head_dim=0), dict(q_heads=9), dict(q_heads=130), dict(cache_format=2), dict(kv_tokens=1 << 31),
    dict(q_tokens=1 << 30), dict(batch=1 << 30), dict(q=(FAKE + 2, 0, 1024, 128)), dict(k=(FAKE, 4, 1024, 128)),
    dict(v=(FAKE, 0, -1024, 128)), dict(out=(0, 0, 1024, 128)), dict(k=(FAKE, 0, 1024, 4)), dict(lse=FAKE + 1),
    dict(lens=FAKE + 2), dict(scale=float("inf"))])
def test_attention_refuses(lib, kw):
    a = attention_args(**kw)
    inv = sz.ERR_INVALID_ARG
    assert lib.splitzip_attention(ctypes.byref(a), FAKE, 1 << 40, None) == inv
    if not set(kw) & {"v", "out"}:
        assert lib.splitzip_attention_weights(ctypes.byref(a), None, FAKE, None) == inv
    if set(kw) & {"batch", "q_tokens", "kv_tokens", "q_heads", "kv_heads", "head_dim", "cache_format"}:
        assert lib.splitzip_attention_workspace_bytes(ctypes.byref(a)) == 0


def test_attention_refuses_its_workspace(lib):
    a = attention_args()
    need = lib.splitzip_attention_workspace_bytes(ctypes.byref(a))
    assert need > 0
    for ws, n in ((None, need), (FAKE + 8, need), (FAKE, need - 1)):
        assert lib.splitzip_attention(ctypes.byref(a), ws, n, None) == sz.ERR_INVALID_ARG
    assert lib.splitzip_attention(None, FAKE, need, None) == sz.ERR_INVALID_ARG
    assert lib.splitzip_attention_workspace_bytes(None) == 0
    for ws in (None, FAKE + 8):
        assert lib.splitzip_attention_status(ws, None) == sz.ERR_INVALID_ARG


def test_attention_weights_refuses_its_buffers(lib):
    inv = sz.ERR_INVALID_ARG
    assert lib.splitzip_attention_weights(ctypes.byref(attention_args()), None, None, None) == inv
    assert lib.splitzip_attention_weights(ctypes.byref(attention_args()), FAKE + 1, FAKE, None) == inv
    assert lib.splitzip_attention_weights(ctypes.byref(attention_args(lse=None)), None, FAKE, None) == inv
    assert lib.splitzip_attention_weights(None, None, FAKE, None) == inv


@pytest.mark.parametrize("kw", [
    dict(head_dim=32), dict(rot_dim=12), dict(rot_dim=136), dict(q_heads=0), dict(kv_heads=0), dict(cache_format=7),
    dict(eps=-1.0), dict(eps=float("nan")), dict(n=1 << 30), dict(positions=None), dict(table=None), dict(slots=None),
    dict(table=FAKE + 4), dict(slots=FAKE + 4), dict(q_weight=FAKE + 8), dict(q=(0, 0, 1024, 128)),
    dict(k=(FAKE, 0, 1023, 128)), dict(k_cache=(FAKE + 8, 0, 1024, 128)), dict(q_out=(FAKE, 0, 1024, -128))])
def test_norm_rope_refuses(lib, kw):
    view = (FAKE, 0, 1024, 128)
    a = serving.NormRopeArgs(view, view, view, None, None, FAKE, FAKE, FAKE, view, view, view, 10, 10, 5, 8, 2, 128, 128,
                             0, 0, 1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.splitzip_qk_norm_rope(ctypes.byref(a), None) == sz.ERR_INVALID_ARG
    assert lib.splitzip_qk_norm_rope(None, None) == sz.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=65536), dict(kv_tokens=0), dict(kv_heads=0), dict(budget=0), dict(head_dim=80),
    dict(keep_first=5, keep_last=4), dict(keep_first=0xFFFFFFFF, keep_last=1), dict(cache_format=3), dict(weights=None),
    dict(index=None), dict(index=FAKE + 2), dict(weights_out=FAKE + 1), dict(k_out=(FAKE, 0, 1024, 4)), dict(v=(0, 0, 0, 0))])
def test_evict_refuses(lib, kw):
    view = (FAKE, 1 << 16, 1024, 128)
    a = serving.EvictArgs(view, view, view, view, FAKE, None, FAKE, None, None, 1, 64, 2, 128, 8, 2, 2, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.splitzip_evict(ctypes.byref(a), None) == sz.ERR_INVALID_ARG
    assert lib.splitzip_evict(None, None) == sz.ERR_INVALID_ARG


def test_workspace_does_not_depend_on_views(lib):
    q = torch.empty((4, 1, 32, 128))
    k = torch.empty((4, 1, 8, 128), dtype=torch.bfloat16).expand(4, 5000, 8, 128)
    assert serving.splitzip_attention_workspace_bytes(q, k) == serving.splitzip_attention_workspace_bytes(q, k.clone())
