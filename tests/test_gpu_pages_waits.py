"""The bounded waits of the paged attention made to run out on purpose (no fault, trap
or hang: one copy of a tile is left out, and what waits for it gives up after a short
limit): the status, NaN for the CTA's rows and nowhere else, and the next call on the
same workspace."""
import ctypes

import pytest
import torch

from lossless_bf16_kv_gb300 import pages as pg
from lossless_bf16_kv_gb300 import serving
from lossless_bf16_kv_gb300 import splitzip as sz
from tests.gpu_helpers import ensure_library
from tests.test_gpu_pages import FORMATS, attend, batch_of

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMIT_MS = 30
NONE = 0xFFFFFFFF


@pytest.fixture(scope="module")
def lib():
    ensure_library()
    return pg.library()


CASES = {  # new tokens, lengths, q_heads, kv_heads: few rows in a cluster of splits, in several clusters, both tiles
    # of a CTA the same rows, two tiles, so many rows that caches are widened first
    "few": ([1, 1], [1500, 1400], 8, 2), "long": ([1], [30000], 4, 1), "tile": ([40, 30], [1200, 1300], 4, 2),
    "tiles": ([120], [900], 8, 2), "many": ([400], [1000], 4, 2),
    "wide": ([1100], [1300], 4, 2)}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("case", list(CASES))
def test_attention_gives_up(lib, case, dim, fmt):
    counts, lens, hq, hk = CASES[case]
    q, p, table, start, lens = batch_of(counts, lens, hq, hk, dim, 16, fmt, seed=dim)
    most = max(counts)
    good, good_lse = attend(q, p, table, start, lens)
    ws = pg.alloc_paged_attention_workspace(q, p, table, most)
    out, lse = torch.zeros_like(q), torch.zeros((hq, q.shape[0]), device=DEV)
    pool = pg.Pool.from_buffer_copy(p.packed)
    a = pg.PagedAttentionArgs((q.data_ptr(), 0, *q.stride()[:2]), (out.data_ptr(), 0, *out.stride()[:2]), pool, lse.data_ptr(),
                              table.data_ptr(), start.data_ptr(), lens.data_ptr(), len(counts), q.shape[0], most,
                              table.shape[1] * 16, table.shape[1], hq, 0, 0, dim ** -0.5)

    def call(cta, tile):
        torch.cuda.synchronize()
        o = serving.WaitTestOpts(LIMIT_MS, cta, tile)
        assert lib.splitzip_paged_attention_test(ctypes.byref(a), ws.data_ptr(), ws.numel(), None, ctypes.byref(o)) == sz.OK
        return serving.splitzip_attention_status(ws)

    some = 0
    for cta, tile in ((0, 0), (1, 1), (2, 3), (3, 2)):
        out.zero_()
        lse.zero_()
        status = call(cta, tile)
        lost = torch.isnan(lse)
        assert status == (sz.ERR_TIMEOUT if bool(lost.any()) else sz.OK)
        some += bool(lost.any())
        assert torch.equal(torch.isnan(out), lost.T[..., None].expand_as(out))
        heads = (lost.any(1).nonzero().flatten() // (hq // hk)).unique()
        assert len(heads) <= 1, "rows of one key/value head"
        assert torch.equal(lse[~lost], good_lse[~lost])
        assert torch.equal(out[~lost.T], good[~lost.T])
    assert some, "no copy was left out"
    assert call(NONE, NONE) == sz.OK
    assert torch.equal(out, good) and torch.equal(lse, good_lse)


def test_the_test_call_refuses(lib):
    q, p, table, start, lens = batch_of([1], [40], 4, 2, 64, 16, "int8", seed=1)
    out = torch.zeros_like(q)
    a = pg.PagedAttentionArgs((q.data_ptr(), 0, *q.stride()[:2]), (out.data_ptr(), 0, *out.stride()[:2]),
                              pg.Pool.from_buffer_copy(p.packed), None, table.data_ptr(), start.data_ptr(), lens.data_ptr(), 1, 1, 1,
                              48, 3, 4, 0, 0, 1.0)
    ws = pg.alloc_paged_attention_workspace(q, p, table, 1)
    long_wait = serving.WaitTestOpts(2001, 0, 0)
    for o in (None, ctypes.byref(long_wait)):
        assert lib.splitzip_paged_attention_test(ctypes.byref(a), ws.data_ptr(), ws.numel(), None, o) == sz.ERR_INVALID_ARG


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
def test_a_piece_of_a_row_tile_gives_up(lib, dim, fmt):
    """160 row tiles, the eight behind a wave of 152 cut into pieces: one that gives up makes its rows NaN, whichever
    piece joins them, and leaves the workspace fit for the next call."""
    q, p, table, start, lens = batch_of([300] * 10, [4000] * 10, 8, 8, dim, 64, fmt, seed=dim)
    good, good_lse = attend(q, p, table, start, lens)
    ws = pg.alloc_paged_attention_workspace(q, p, table, 300)
    out, lse = torch.zeros_like(q), torch.zeros((8, q.shape[0]), device=DEV)
    pool = pg.Pool.from_buffer_copy(p.packed)
    a = pg.PagedAttentionArgs((q.data_ptr(), 0, *q.stride()[:2]), (out.data_ptr(), 0, *out.stride()[:2]), pool, lse.data_ptr(),
                              table.data_ptr(), start.data_ptr(), lens.data_ptr(), 10, q.shape[0], 300,
                              table.shape[1] * 64, table.shape[1], 8, 0, 0, dim ** -0.5)

    def call(cta, tile):
        torch.cuda.synchronize()
        o = serving.WaitTestOpts(LIMIT_MS, cta, tile)
        assert lib.splitzip_paged_attention_test(ctypes.byref(a), ws.data_ptr(), ws.numel(), None, ctypes.byref(o)) == sz.OK
        return serving.splitzip_attention_status(ws)

    some = 0
    for cta in (152, 156, 171):
        out.zero_()
        lse.zero_()
        status = call(cta, 1)
        lost = torch.isnan(lse)
        assert status == (sz.ERR_TIMEOUT if bool(lost.any()) else sz.OK)
        some += bool(lost.any())
        assert torch.equal(torch.isnan(out), lost.T[..., None].expand_as(out))
        assert len(lost.any(1).nonzero()) <= 1, "rows of one head"
        assert int(lost.sum()) <= 256, "rows of one row tile"
        assert torch.equal(lse[~lost], good_lse[~lost])
        assert torch.equal(out[~lost.T], good[~lost.T])
    assert some == 3, "no copy was left out"
    assert call(NONE, NONE) == sz.OK
    assert torch.equal(out, good) and torch.equal(lse, good_lse)
