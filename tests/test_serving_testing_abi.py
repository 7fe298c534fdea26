"""include/splitzip_serving_testing.h on the CPU: plain C, exported, bound, and
refusing what it cannot do."""
import ctypes
import os
import re
import subprocess

import pytest

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
