"""The bounded waits of the tensor-core kernels made to run out on purpose (no fault,
trap or hang: one copy of a tile is left out, and what waits for it gives up after
a short limit): the status, NaN where there is no result and nowhere else, and the
next call on the same workspace."""
import ctypes

import pytest
import torch

from lossless_bf16_kv_gb300 import serving
from lossless_bf16_kv_gb300 import splitzip as sz
from tests.gpu_helpers import ensure_library
from tests.test_gpu_serving import attend, make

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMIT_MS = 30
NONE = 0xFFFFFFFF


@pytest.fixture(scope="module")
def lib():
    ensure_library()
    return serving.library()


def arguments(q, kv, out, lse, window=0):
    view = lambda t: (t.data_ptr(), *t.stride()[:3]) if t is not None else (0, 0, 0, 0)  # noqa: E731
    b, tq, hq, d = q.shape
    return serving.AttentionArgs(view(q), view(kv[:, 0]), view(kv[:, 1]), view(out), lse.data_ptr(), None, b, tq, kv.shape[2], hq,
                                 kv.shape[3], d, window, 0, 0 if kv.dtype == torch.bfloat16 else 1, d ** -0.5)


def opts(cta, tile, ms=LIMIT_MS):
    return ctypes.byref(serving.WaitTestOpts(ms, cta, tile))


SHAPES = [  # more row tiles than one with a split each, clusters of splits, both tiles of a CTA the same rows
    (4, 1100, 1100, 24, 3, 128, 0), (4, 1100, 1100, 24, 3, 64, 200), (1, 300, 4000, 4, 2, 128, 0), (1, 300, 4000, 4, 2, 64, 0),
    (2, 40, 3000, 8, 2, 128, 0), (2, 40, 3000, 8, 2, 64, 0)]


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("tile", [0, 1, 2, 5])
@pytest.mark.parametrize("shape", SHAPES)
def test_attention_gives_up(lib, shape, tile, fmt):
    b, tq, tk, hq, hk, d, window = shape
    q, kv = make(*shape[:6], fmt=fmt, seed=tile)
    good, good_lse = attend(q, kv, None, window)
    ws = serving.alloc_attention_workspace(q, kv[:, 0], window)
    out = torch.zeros_like(q)
    lse = torch.zeros((b, hq, tq), device=DEV)
    a = arguments(q, kv, out, lse, window)
    call = lambda o: lib.splitzip_attention_test(ctypes.byref(a), ws.data_ptr(), ws.numel(), None, o)  # noqa: E731
    torch.cuda.synchronize()
    group = hq // hk
    rows = 2 * (128 // group)        # query tokens of a CTA's two tiles
    assert call(opts(3, tile)) == sz.OK
    assert serving.splitzip_attention_status(ws) == sz.ERR_TIMEOUT
    assert serving.splitzip_attention_status(ws) == sz.OK      # reported once
    lost = torch.isnan(lse)
    assert torch.equal(torch.isnan(out), lost.transpose(1, 2)[..., None].expand_as(out))
    # All rows of one row tile of one head, and no others.
    assert bool(lost.any())
    where = lost.nonzero()
    assert len(where[:, 0].unique()) == 1 and len((where[:, 1] // group).unique()) == 1
    tokens = where[:, 2].unique()
    first = int(tokens[0]) // rows * rows
    assert tokens.tolist() == list(range(first, min(first + rows, tq))) and len(where) == group * len(tokens)
    keep = ~lost
    assert torch.equal(lse[keep], good_lse[keep])
    assert torch.equal(out[keep.transpose(1, 2)], good[keep.transpose(1, 2)])
    # The same workspace, nothing left out: all there, and to the bit.
    assert call(opts(NONE, NONE)) == sz.OK
    assert serving.splitzip_attention_status(ws) == sz.OK
    assert torch.equal(out, good) and torch.equal(lse, good_lse)


def test_attention_without_waits_is_refused(lib):
    q, kv = make(1, 1, 300, 8, 2, 128)
    ws = serving.alloc_attention_workspace(q, kv[:, 0])
    a = arguments(q, kv, torch.empty_like(q), torch.empty((1, 8, 1), device=DEV))
    assert lib.splitzip_attention_test(ctypes.byref(a), ws.data_ptr(), ws.numel(), None, opts(0, 0)) == sz.ERR_INVALID_ARG
    assert lib.splitzip_attention_test(ctypes.byref(a), ws.data_ptr(), ws.numel(), None, None) == sz.ERR_INVALID_ARG


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tq,cta,tile", [(600, 0, 0), (600, 3, 1), (600, 7, 9), (600, 50, 14), (600, 50, 22), (600, 151, 30),
                                         (600, 20, 37), (30, 0, 0), (30, 9, 1), (30, 40, 3), (30, 41, 4), (100, 40, 3), (100, 77, 5)])
def test_weights_give_up(lib, tq, cta, tile, dim, fmt):
    """NaN for the item of 128 slots that the tile belongs to and for those after it that
    the CTA had left; the others are right, to the bit."""
    b, tk, hq, hk = 8, 2500, 16, 8
    q, kv = make(b, tq, tk, hq, hk, dim, fmt=fmt, seed=tile)
    _, lse = attend(q, kv, None)
    before = torch.rand((b, hk, tk), device=DEV)
    good, got = torch.empty_like(before), torch.zeros_like(before)
    a = arguments(q, kv, None, lse)
    call = lambda o, w: lib.splitzip_attention_weights_test(ctypes.byref(a), before.data_ptr(), w.data_ptr(), None, o)  # noqa: E731
    torch.cuda.synchronize()
    assert call(opts(NONE, NONE), good) == sz.OK
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    tiles, heads = -(-tk // 128), b * hk
    assert tiles * heads > 3 * ctas
    mine = [at for i in range(-(-tiles * heads // ctas)) if (at := i * ctas + (ctas - 1 - cta if i % 2 else cta)) < tiles * heads]
    for _ in range(3):
        got.zero_()
        torch.cuda.synchronize()
        assert call(opts(cta, tile), got) == sz.OK
        torch.cuda.synchronize()
        lost = torch.isnan(got)
        state = []
        for at in mine:
            sc, bh = divmod(at, heads)
            part = lost[bh // hk, bh % hk, sc * 128:(sc + 1) * 128]
            assert bool(part.all()) or not bool(part.any())
            state.append(bool(part.any()))
        assert any(state) and state == sorted(state), state            # from one item on
        assert int(lost.sum()) == sum(min(128, tk - at // heads * 128) for at, s in zip(mine, state) if s)
        assert torch.equal(got[~lost], good[~lost])
    # How many tiles come before the lost item: none of them was the one left out.
    seen = 0
    for at, s in zip(mine, state):
        s_lo, first = at // heads * 128, tk - tq
        t_lo = max(0, s_lo - first)
        i0 = t_lo // 64
        count = 1 + (-(-tq // 64) - i0) if t_lo < tq else 0
        if s:
            assert seen <= tile < seen + count
            break
        seen += count
    assert call(opts(NONE, NONE), got) == sz.OK
    assert torch.equal(got, good)
