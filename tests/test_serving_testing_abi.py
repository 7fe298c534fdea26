"""include/splitzip_serving_testing.h on the CPU: plain C, exported, bound, and
refusing what it cannot do."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from lossless_bf16_kv_gb300 import _build, serving
from lossless_bf16_kv_gb300 import splitzip as sz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20   # aligned, never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return serving.library()


def test_exports_and_binds_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "splitzip_serving_testing.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(splitzip_\w+)\s*\(", text)))
    assert names == ["splitzip_attention_test", "splitzip_attention_weights_test"]
    for name in names:
        assert getattr(lib, name).argtypes is not None, name


def test_options_have_the_c_layout(tmp_path):
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "splitzip_serving_testing.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu", sizeof(splitzip_wait_test_opts), offsetof(splitzip_wait_test_opts, wait_ms),'
                   ' offsetof(splitzip_wait_test_opts, cta), offsetof(splitzip_wait_test_opts, tile));\nreturn 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    o = serving.WaitTestOpts
    assert got == [ctypes.sizeof(o), o.wait_ms.offset, o.cta.offset, o.tile.offset]


def test_refusals(lib):
    view = (FAKE, 1 << 20, 1 << 10, 128)
    a = serving.AttentionArgs(view, view, view, view, FAKE, None, 2, 300, 640, 8, 2, 128, 0, 0, 0, 1.0)
    few = serving.AttentionArgs(view, view, view, view, FAKE, None, 2, 1, 640, 8, 2, 128, 0, 0, 0, 1.0)
    bad = serving.AttentionArgs(view, view, view, view, FAKE, None, 2, 300, 640, 9, 2, 128, 0, 0, 0, 1.0)
    fine, long = serving.WaitTestOpts(10, 0, 0), serving.WaitTestOpts(2001, 0, 0)
    inv = sz.ERR_INVALID_ARG
    for args, o in ((a, None), (a, ctypes.byref(long)), (few, ctypes.byref(fine)), (bad, ctypes.byref(fine))):
        assert lib.splitzip_attention_test(ctypes.byref(args), FAKE, 1 << 40, None, o) == inv
    for args, o in ((a, None), (a, ctypes.byref(long)), (bad, ctypes.byref(fine))):
        assert lib.splitzip_attention_weights_test(ctypes.byref(args), None, FAKE, None, o) == inv


@pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call would run; here it ends at the missing GPU")
@pytest.mark.parametrize("fmt,dim,units,rows,tiles", [
    (0, 128, 128, 16, False), (0, 128, 128, 24, True), (0, 64, 16, 24, True),
    (1, 128, 128, 32, False), (1, 128, 128, 40, True), (1, 128, 24, 64, True), (1, 128, 512, 40, True),      # 265 us against 278
    (1, 128, 16, 64, False), (1, 64, 128, 64, False), (1, 64, 16, 64, False), (1, 64, 128, 128, True), (1, 128, 16, 72, True)])
def test_kernel_by_rows_and_units(lib, fmt, dim, units, rows, tiles):
    """Which of the two attention kernels takes a call, on both sides of the rule's
    limits: the test entry refuses the one without waits."""
    view = (FAKE, 1 << 24, 1 << 10, 128)
    a = serving.AttentionArgs(view, view, view, view, FAKE, None, units, 1, 2048, rows, 1, dim, 0, 0, fmt, 1.0)
    if rows > 64:
        a.q_tokens, a.q_heads = rows // 8, 8
    got = lib.splitzip_attention_test(ctypes.byref(a), FAKE, 1 << 40, None, ctypes.byref(serving.WaitTestOpts(10, 0, 0)))
    assert got == (sz.ERR_CUDA if tiles else sz.ERR_INVALID_ARG)
