"""include/splitzip_pages.h on the CPU: its functions are exported and bound, the
binding's structures have the C ones' layout, and every argument that the host
checks refuse is refused before anything is enqueued (no GPU is needed to see
that)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from lossless_bf16_kv_gb300 import _build
from lossless_bf16_kv_gb300 import pages as pg
from lossless_bf16_kv_gb300 import splitzip as sz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "splitzip_pages.h")
STRUCTS = {"splitzip_page_rows": pg.PageRows, "splitzip_pool": pg.Pool, "splitzip_pages_store_args": pg.PagesStoreArgs,
           "splitzip_pages_load_args": pg.PagesLoadArgs, "splitzip_paged_attention_args": pg.PagedAttentionArgs}
INV = sz.ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return pg.library()


def test_library_exports_and_binds_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(splitzip_\w+)\s*\(", text)))
    assert len(names) == 4
    for name in names:
        assert getattr(lib, name).argtypes is not None, name


def test_structures_have_the_c_layout(tmp_path):
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("%zu ", sizeof({name}));')
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu ", offsetof({name}, {f}));')
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "splitzip_pages.h"\nint main(void) {\n'
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
    assert [x.size for x in (pg._POOL, pg._STORE, pg._LOAD, pg._ATTENTION)] == \
        [ctypes.sizeof(x) for x in (pg.Pool, pg.PagesStoreArgs, pg.PagesLoadArgs, pg.PagedAttentionArgs)]


FAKE = 1 << 20   # aligned, never dereferenced: every call below is refused
VIEW = (FAKE, 1 << 20, 1 << 10, 128)
ROWS = (FAKE, 1 << 14, 1 << 10, 128, FAKE, 1 << 10, 32, 4)


def pool_of(**kw):
    p = pg.Pool(ROWS, ROWS, 10, 16, 8, 128, pg.INT8)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def calls(lib, pool, **kw):
    """Status of each of the three calls with this pool."""
    store = pg.PagesStoreArgs(VIEW, VIEW, FAKE, pool, 4)
    load = pg.PagesLoadArgs(pool, FAKE, FAKE, VIEW, VIEW, 2, 48, 3, pg.BF16)
    att = pg.PagedAttentionArgs(VIEW, VIEW, pool, FAKE, FAKE, FAKE, FAKE, 2, 6, 4, 48, 3, 32, 0, 0, 1.0)
    found = {}
    for name, a in (("store", store), ("load", load), ("attention", att)):
        mine = {k[len(name) + 1:]: v for k, v in kw.items() if k.startswith(name + "_")}
        if kw and not mine:
            continue
        for k, v in mine.items():
            setattr(a, k, v)
        if name == "attention":
            found[name] = lib.splitzip_paged_attention(ctypes.byref(a), FAKE, 1 << 40, None)
        else:
            found[name] = getattr(lib, f"splitzip_pages_{name}")(ctypes.byref(a), None)
    return found


@pytest.mark.parametrize("kw", [
    dict(pages=0), dict(pages=1 << 31), dict(page_tokens=0), dict(page_tokens=8), dict(page_tokens=24),
    dict(page_tokens=1 << 17), dict(kv_heads=0), dict(head_dim=96), dict(head_dim=0), dict(format=4),
    dict(k=(0, *ROWS[1:])), dict(v=(FAKE + 8, *ROWS[1:])), dict(k=(FAKE, 8, *ROWS[2:])), dict(v=(FAKE, 1 << 14, 0, *ROWS[3:])),
    dict(k=(FAKE, 1 << 14, -1024, *ROWS[3:])), dict(k=(*ROWS[:3], 100, *ROWS[4:])), dict(v=(FAKE, 1 << 38, *ROWS[2:])),
    dict(k=(*ROWS[:4], 0, *ROWS[5:])), dict(v=(*ROWS[:4], FAKE + 2, *ROWS[5:])), dict(k=(*ROWS[:5], 0, 32, 4)),
    dict(v=(*ROWS[:6], 6, 4)), dict(k=(*ROWS[:7], 2)), dict(format=pg.E2M1, k=(FAKE, 1 << 14, 1 << 10, 24, *ROWS[4:]))])
def test_every_call_refuses_these_pools(lib, kw):
    assert set(calls(lib, pool_of(**kw)).values()) == {INV}


@pytest.mark.parametrize("kw", [
    dict(store_k=(0, 0, 1024, 128)), dict(store_v=(FAKE + 2, 0, 1024, 128)), dict(store_k=(FAKE, 0, 1020, 128)),
    dict(store_v=(FAKE, 0, 0, 128)), dict(store_slots=0), dict(store_slots=FAKE + 4), dict(store_n=1 << 29),
    dict(load_table=0), dict(load_table=FAKE + 2), dict(load_lens=FAKE + 1), dict(load_k_out=(0, *VIEW[1:])),
    dict(load_k_out=(FAKE, 0, 1 << 10, 128)), dict(load_v_out=(FAKE, 1 << 20, 4, 128)), dict(load_batch=0), dict(load_tokens=0),
    dict(load_tokens=49), dict(load_tokens=1 << 31), dict(load_out_format=pg.E5M2), dict(load_out_format=pg.INT8),
    dict(load_batch=1 << 28), dict(attention_batch=0), dict(attention_tokens=0), dict(attention_max_q_tokens=0),
    dict(attention_max_q_tokens=7), dict(attention_kv_tokens=0), dict(attention_kv_tokens=49), dict(attention_q_heads=0),
    dict(attention_q_heads=12), dict(attention_q_heads=65 * 8), dict(attention_scale=0.0), dict(attention_scale=-1.0),
    dict(attention_scale=float("inf")), dict(attention_scale=float("nan")), dict(attention_table=0),
    dict(attention_q_start=0), dict(attention_lens=0), dict(attention_q_start=FAKE + 2), dict(attention_lse=FAKE + 2),
    dict(attention_q=(0, 0, 1024, 128)), dict(attention_q=(FAKE, 0, 1024, 4)), dict(attention_out=(FAKE + 4, 0, 1024, 128)),
    dict(attention_out=(FAKE, 0, 0, 128)), dict(attention_batch=1 << 28), dict(attention_tokens=1 << 30)])
def test_a_call_refuses(lib, kw):
    assert set(calls(lib, pool_of(), **kw).values()) == {INV}


def test_attention_refuses_a_small_or_crooked_workspace(lib):
    a = pg.PagedAttentionArgs(VIEW, VIEW, pool_of(), FAKE, FAKE, FAKE, FAKE, 2, 6, 4, 48, 3, 32, 0, 0, 1.0)
    need = lib.splitzip_paged_attention_workspace_bytes(ctypes.byref(a))
    assert need >= 1024
    for ws, size in ((None, need), (FAKE + 8, need), (FAKE, need - 1)):
        assert lib.splitzip_paged_attention(ctypes.byref(a), ws, size, None) == INV
    a.kv_tokens = 49
    assert lib.splitzip_paged_attention_workspace_bytes(ctypes.byref(a)) == 0
    for fn in (lib.splitzip_pages_store, lib.splitzip_pages_load):
        assert fn(None, None) == INV
    assert lib.splitzip_paged_attention(None, FAKE, 1 << 40, None) == INV


def test_store_of_no_tokens_enqueues_nothing(lib):
    a = pg.PagesStoreArgs((0, 0, 0, 0), (0, 0, 0, 0), 0, pool_of(), 0)
    assert lib.splitzip_pages_store(ctypes.byref(a), None) == sz.OK


def test_workspace_grows_to_what_many_splits_need(lib):
    a = pg.PagedAttentionArgs(VIEW, VIEW, pool_of(kv_heads=1, pages=1 << 20), 0, 0, 0, 0, 1, 1, 1, 1 << 17, 1 << 13, 4, 0, 0, 1.0)
    few = pg.PagedAttentionArgs(VIEW, VIEW, pool_of(kv_heads=1, pages=1 << 20), 0, 0, 0, 0, 1, 1, 1, 128, 1 << 13, 4, 0, 0, 1.0)
    assert lib.splitzip_paged_attention_workspace_bytes(ctypes.byref(a)) > \
        lib.splitzip_paged_attention_workspace_bytes(ctypes.byref(few))


# ----------------------------------------------------- the binding's checks

def refused(fn, *args, **kw):
    with pytest.raises((pg.SplitZipError, ValueError)) as e:
        fn(*args, **kw)
    assert getattr(e.value, "status", INV) == INV


def test_a_pool_refuses_what_is_none(lib):
    rows = torch.zeros((4, 16, 2, 128), dtype=torch.int8)
    exps = torch.zeros((4, 16, 2, 4), dtype=torch.uint8)
    for args in ((rows.float(), rows.float()), (rows, rows.view(torch.uint8)), (rows, rows), (rows, rows, exps),
                 (rows, rows, exps.short(), exps), (rows, rows, exps[:3], exps), (rows[0], rows[0], exps, exps),
                 (rows.bfloat16(), rows.bfloat16(), exps, exps), (rows, rows[:3], exps, exps),
                 (rows, rows, exps, exps)):     # the last: not on a GPU
        refused(pg.Pages, *args)
    refused(pg.alloc_pages, 4, 16, 2, 128, "fp8", "cpu")


class FakePages:
    """What the binding's checks look at, without a GPU."""
    k = torch.zeros(1)
    format, pages, page_tokens, kv_heads, head_dim, index, packed = pg.INT8, 4, 16, 2, 128, 0, bytes(152)


def test_the_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    p = FakePages()
    rows = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    for k, v, s in ((rows, rows, slots), (rows.float(), rows, slots), (rows, rows[:2], slots), (rows[:, :1], rows[:, :1], slots),
                    (rows, rows, slots[:2]), (rows, rows, slots.int())):
        refused(pg.splitzip_pages_store, k, v, s, p)
    out = torch.zeros((2, 40, 2, 128), dtype=torch.bfloat16)
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for args in ((table, lens, out, out), (table, lens, out.float(), out), (table, lens, out, out[:1]),
                 (table.long(), lens, out, out), (table[:1], lens, out, out), (table[:, :2], lens, out, out),
                 (table, lens[:1], out, out), (table, lens, out.to(torch.float8_e5m2), out.to(torch.float8_e5m2))):
        refused(pg.splitzip_pages_load, p, *args)
    q, start, ws = torch.zeros((5, 4, 128), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32), torch.zeros(2048, dtype=torch.uint8)
    good = dict(q=q, pages=p, table=table, q_start=start, lens=lens, out=q, workspace=ws, max_q_tokens=2)
    for kw in ({}, dict(q=q.float()), dict(out=q[:4]), dict(q_start=start[:2]), dict(lens=lens[:1]), dict(max_q_tokens=0),
               dict(max_q_tokens=6), dict(kv_tokens=49), dict(kv_tokens=-1), dict(window=-1), dict(workspace=ws.int()),
               dict(lse=torch.zeros((5, 4)))):
        refused(pg.splitzip_paged_attention, **{**good, **kw})
    assert pg.splitzip_paged_attention_workspace_bytes(q, p, table, 0) == 0


class Here(torch.Tensor):
    """A tensor that says that it lies on GPU 0."""
    is_cuda = True

    def get_device(self):
        return 0


class There(Here):
    def get_device(self):
        return 1


def test_tensors_of_another_device_are_refused(lib, monkeypatch):
    """Every tensor of a call in turn on the other GPU; with all of them on the current one the call is made."""
    def zeros(dtype, *shape):
        return torch.zeros(shape, dtype=dtype).as_subclass(Here)
    calls = []
    for module in (pg, pg._sz):
        monkeypatch.setattr(module, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(pg, "_stream_of", lambda s: 0)
    for name in ("_fn_store", "_fn_load", "_fn_attention"):
        monkeypatch.setattr(pg, name, lambda *a: calls.append(a) or 0)
    bf16, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    rows = {"k": zeros(torch.int8, 4, 16, 2, 64), "v": zeros(torch.int8, 4, 16, 2, 64),
            "k_exp": zeros(u8, 4, 16, 2, 4), "v_exp": zeros(u8, 4, 16, 2, 4)}
    p = pg.Pages(**rows)
    for name in ("v", "k_exp", "v_exp"):
        monkeypatch.setattr(There, "device", torch.device("cuda:1"), raising=False)
        with pytest.raises(sz.SplitZipError):
            pg.Pages(**{**rows, name: rows[name].as_subclass(There)})
    store = {"k": zeros(bf16, 5, 2, 64), "v": zeros(bf16, 5, 2, 64), "slots": zeros(torch.int64, 5)}
    load = {"table": zeros(i32, 3, 2), "lens": zeros(i32, 3), "k_out": zeros(bf16, 3, 30, 2, 64), "v_out": zeros(bf16, 3, 30, 2, 64)}
    attend = {"q": zeros(bf16, 5, 4, 64), "table": zeros(i32, 3, 2), "q_start": zeros(i32, 4), "lens": zeros(i32, 3),
              "out": zeros(bf16, 5, 4, 64), "workspace": zeros(u8, 1 << 16), "lse": zeros(torch.float32, 4, 5)}
    for fn, args, more in ((pg.splitzip_pages_store, store, {}), (pg.splitzip_pages_load, load, {}),
                           (pg.splitzip_paged_attention, attend, {"max_q_tokens": 3})):
        calls.clear()
        fn(pages=p, **args, **more)
        assert len(calls) == 1
        for name in args:
            with pytest.raises(sz.SplitZipError):
                fn(pages=p, **{**args, name: args[name].as_subclass(There)}, **more)
        assert len(calls) == 1, fn.__name__


def test_a_pool_whose_memory_has_moved_is_refused(lib, monkeypatch):
    """A handle holds addresses: of tensors resized since, memory that is no longer theirs."""
    def zeros(dtype, *shape):
        return torch.zeros(shape, dtype=dtype).as_subclass(Here)
    made = []
    monkeypatch.setattr(pg, "_current_device", lambda: 0)
    monkeypatch.setattr(pg, "_stream_of", lambda s: 0)
    for name in ("_fn_store", "_fn_load", "_fn_attention"):
        monkeypatch.setattr(pg, name, lambda *a: made.append(a) or 0)
    bf16, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    new, table, ints = zeros(bf16, 5, 2, 64), zeros(i32, 3, 2), zeros(i32, 3)

    def every_call(p):
        yield lambda: pg.splitzip_pages_store(new, new, zeros(torch.int64, 5), p)
        yield lambda: pg.splitzip_pages_load(p, table, ints, zeros(bf16, 3, 30, 2, 64), zeros(bf16, 3, 30, 2, 64))
        yield lambda: pg.splitzip_paged_attention(zeros(bf16, 5, 4, 64), p, table, zeros(i32, 4), ints, zeros(bf16, 5, 4, 64),
                                                  zeros(u8, 1 << 16), 3)

    def fresh():
        return {"k": zeros(torch.int8, 4, 16, 2, 64), "v": zeros(torch.int8, 4, 16, 2, 64), "k_exp": zeros(u8, 4, 16, 2, 4),
                "v_exp": zeros(u8, 4, 16, 2, 4)}
    for name in ("k", "v", "k_exp", "v_exp"):
        rows = fresh()
        p = pg.Pages(**rows)
        with pytest.raises(AttributeError):
            setattr(p, name, rows[name].clone())
        # What changes the caller's tensor alone leaves the pool as it is.
        rows[name].transpose_(0, 1)
        made.clear()
        for call in every_call(p):
            call()
        assert len(made) == 3 and getattr(p, name).shape[:3] == (4, 16, 2)
        rows[name].untyped_storage().resize_(1 << 20)
        for call in every_call(p):
            with pytest.raises(sz.SplitZipError) as e:
                call()
            assert e.value.status == INV
        assert len(made) == 3


@pytest.mark.parametrize("heads,few", [(8, True), (16 * 8, True), (17 * 8, False), (64 * 8, False)])
@pytest.mark.parametrize("tokens", [16, 40])
def test_no_few_row_kernel_where_a_token_has_too_many_rows(lib, heads, few, tokens):
    """16 sequences of 16k in 8 bits: where a single token has up to 16 query rows the few-row kernel may have to share
    their work out, whose partial results take megabytes; where it has more, that kernel has no sequence."""
    pool = pool_of(pages=1 << 20)
    a = pg.PagedAttentionArgs(VIEW, VIEW, pool, 0, 0, 0, 0, 16, tokens, 1, 16384, 1024, heads, 0, 0, 1.0)
    size = lib.splitzip_paged_attention_workspace_bytes(ctypes.byref(a))
    assert size > 1 << 20 if few else size == 1024


def test_a_table_of_more_slots_than_a_sequence_may_have(lib, monkeypatch):
    """Without kv_tokens the bound is what the table holds, or the most that a call takes."""
    def zeros(dtype, *shape):
        return torch.zeros(shape, dtype=dtype).as_subclass(Here)
    made = []
    monkeypatch.setattr(pg, "_current_device", lambda: 0)
    monkeypatch.setattr(pg, "_stream_of", lambda s: 0)
    monkeypatch.setattr(pg, "_fn_attention", lambda a, *more: made.append(pg.PagedAttentionArgs.from_buffer_copy(a)) or 0)
    i32 = torch.int32
    rows, exps = zeros(torch.int8, 1, 65536, 1, 64), zeros(torch.uint8, 1, 65536, 1, 4)
    p = pg.Pages(rows, rows, exps, exps)
    q, ws = zeros(torch.bfloat16, 3, 4, 64), zeros(torch.uint8, 1 << 16)
    for width, most in ((1, 65536), ((1 << 15) - 1, 65536 * ((1 << 15) - 1)), (1 << 15, (1 << 31) - 256), (1 << 17, (1 << 31) - 256)):
        table = zeros(i32, 1, width)
        size = pg.splitzip_paged_attention_workspace_bytes(q, p, table, 3)
        assert size and size == pg.splitzip_paged_attention_workspace_bytes(q, p, table, 3, most)
        pg.splitzip_paged_attention(q, p, table, zeros(i32, 2), zeros(i32, 1), q.clone(), ws, 3)
        assert made[-1].kv_tokens == most
    assert pg.splitzip_paged_attention_workspace_bytes(q, p, table, 3, (1 << 31) - 255) == 0
