"""Attention of so many new tokens that quantised and E5M2 caches are widened ahead of the products."""
import ctypes

import pytest
import torch

from lossless_bf16_kv_gb300 import pages as pg
from lossless_bf16_kv_gb300 import serving
from lossless_bf16_kv_gb300 import splitzip as sz
from tests import pages_ref, serving_ref
from tests.gpu_helpers import ensure_library
from tests.test_gpu_pages import DEV, attend, batch_of, close, ints

pytestmark = pytest.mark.gpu
WIDENED = ["e5m2", "int8", "e2m1"]


@pytest.fixture(autouse=True)
def _built():
    ensure_library()


def ones_of_either_sign(p, fmt):
    """Values 1 in even slots of a page and -1 in odd ones."""
    neg = torch.arange(p.page_tokens, device=DEV)[None, :, None, None] % 2 == 1
    one = {"int8": (64, -64, 121), "e2m1": (0x22, 0xAA, 127), "e5m2": (1.0, -1.0, None)}[fmt]
    p.v.copy_(torch.where(neg, one[1], one[0]).expand(p.v.shape).to(p.v.dtype))
    if p.v_exp is not None:
        p.v_exp.fill_(one[2])


@pytest.mark.parametrize("fmt", WIDENED)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("counts", [[200], [600], [600, 1, 220, 530]], ids=["tiles", "widened", "both"])
def test_weights_keep_eleven_bits(counts, dim, fmt):
    """Queries that see two slots, with values 1 and -1: the output is the difference of two weights, and where they are
    nearly alike it shows their rounding.  FP16 weights are off by at most 2^-11 of their sum, the output's own rounding
    is 2^-8 of it; 2^-13 and the scores' errors (which the bound of lse has) are serving_ref's."""
    lens = [n + 150 for n in counts]
    q, p, table, start, lens = batch_of(counts, lens, 8, 2, dim, 16, fmt, seed=dim)
    ones_of_either_sign(p, fmt)
    out, lse = attend(q, p, table, start, lens, window=2)
    near = 0
    for b, n in enumerate(lens.tolist()):
        i, j = start[b].item(), start[b + 1].item()
        k, v = (pages_ref.sequence(p, table[b], n, x)[None] for x in "kv")
        o, l, _, ltol = serving_ref.attention(q[None, i:j], k, v, ints([n]), 2, 0, dim ** -0.5)
        tol = o[0].abs() * 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13 + 2 * ltol[0].T[..., None]
        near += int((o.abs() < 2.0 ** -4).sum())
        close(out[i:j], o[0], tol, "out")
        close(lse[:, i:j], l[0], ltol[0], "lse")
    assert near > 1000


def widened_caches(ws, kv_tokens, p, fmt, batch, rows):
    """[sequences, k and v, heads, tokens, dim] in FP16, which lie at the workspace's end: of as many sequences as `rows`
    query rows may be widened for (from 1025 on, or 2049)."""
    border = 2048 if fmt == "e5m2" and p.head_dim == 128 else 1024
    sequences = 1 if batch == 1 else min(batch, rows // (border + 1))
    shape = (sequences, 2, p.kv_heads, -(-kv_tokens // 128) * 128, p.head_dim)
    count = torch.Size(shape).numel()
    return ws[ws.numel() - 2 * count:].view(torch.float16).view(shape)


@pytest.mark.parametrize("fmt", WIDENED)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3), (300, 200)])
@pytest.mark.parametrize("lens", [[777], [1290, 5, 601, 700], [1281, 610, 640, 0]], ids=["one", "three", "ends"])
def test_widened_caches_hold_nothing_of_the_workspace(lens, window, sinks, dim, fmt):
    """Where queries look at tiles of 128 slots, those are the pool's rows and zeros, whatever lay there before: NaN of
    another call would be kept out of the products value by value."""
    counts = [600 if n > 600 else 0 for n in lens]
    q, p, table, start, lens = batch_of(counts, lens, 8, 2, dim, 16, fmt, seed=dim)
    kv_tokens = table.shape[1] * 16
    ws = pg.alloc_paged_attention_workspace(q, p, table, 600, None, window, sinks)
    wide = widened_caches(ws, kv_tokens, p, fmt, len(counts), 4 * len(q))
    wide.fill_(float("nan"))
    out, lse = attend(q, p, table, start, lens, most=600, window=window, sinks=sinks, ws=ws)
    for rows, o, l, tol, ltol in pages_ref.attention(q, p, table, start, lens, kv_tokens, window, sinks, dim ** -0.5):
        close(out[rows], o, tol, "out")
        close(lse[:, rows], l, ltol, "lse")
    for rank, b in enumerate(b for b, n in enumerate(counts) if n):
        n = lens[b].item()
        t = torch.arange(wide.shape[3], device=DEV)
        first = n - counts[b] - window + 1 if window else 0                  # of the first query's window
        looked_at = (t // 128 * 128 < n) & ((t // 128 * 128 + 128 > first) | (t // 128 * 128 < sinks))
        seen = (t < n) & ((t >= first) | (t < sinks))
        for i, x in enumerate("kv"):
            rows = pages_ref.sequence(p, table[b], n, x)
            got = wide[rank, i].transpose(0, 1).double()
            assert torch.equal(got[:n][seen[:n]], rows[seen[:n]])
            others = got[looked_at & ~seen]
            assert not others.isnan().any()
            assert not got[looked_at & (t >= n)].any()


#: new tokens of three sequences, whose row tiles (eight heads of four query heads) are waves of 152 and some more that
#: are cut: of the widened sequences, of the others, of both, which run at the same time
CUT = [[600, 600, 600], [600, 250, 250], [320, 256, 250], [600, 200, 1], [250, 250, 250], [0, 600, 30]]


@pytest.mark.parametrize("fmt", WIDENED)
@pytest.mark.parametrize("dim", [64, 128])
def test_pieces_of_widened_and_other_row_tiles_at_once(dim, fmt):
    """Both tile launches of a call cut their last waves, each with counters and partial results of its own."""
    q, p, table, _, lens = batch_of([600] * 3, [8000, 7900, 7000], 32, 8, dim, 64, fmt, seed=dim)
    ws = pg.alloc_paged_attention_workspace(q, p, table, 600)
    sequences = min(3, 4 * len(q) // (2049 if fmt == "e5m2" and dim == 128 else 1025))
    pieces = 202 * (dim // 4 + 1) * 256 * 16                                 # bytes, of a launch that is cut
    rest = ws.numel() - sequences * 8064 * 8 * dim * 4 - 2 * pieces
    assert 0 < rest < pieces, "partial results of two launches"
    scale = dim ** -0.5
    for counts in CUT:
        start = ints([0, *torch.tensor(counts).cumsum(0).tolist()])
        out, lse = attend(q, p, table, start, lens, most=600, ws=ws)
        for rows, o, l, tol, ltol in pages_ref.attention(q, p, table, start, lens, table.shape[1] * 64, 0, 0, scale):
            close(out[rows], o, tol, "out")
            close(lse[:, rows], l, ltol, "lse")
        assert bool((out[sum(counts):] == 7.0).all()) and bool((lse[:, sum(counts):] == 7.0).all())
        for _ in range(3):
            again = attend(q, p, table, start, lens, most=600, ws=ws)
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("fmt", WIDENED)
@pytest.mark.parametrize("dim", [64, 128])
def test_a_piece_of_a_widened_row_tile_gives_up(dim, fmt):
    """240 row tiles of widened sequences, the 88 behind a wave of 152 cut: a copy that is left out of a piece makes the
    row tile's rows NaN, whichever piece joins them, and leaves the workspace fit for the next call."""
    q, p, table, start, lens = batch_of([600] * 3, [8000, 7900, 7000], 32, 8, dim, 64, fmt, seed=dim + 1)
    good, good_lse = attend(q, p, table, start, lens)
    ws = pg.alloc_paged_attention_workspace(q, p, table, 600)
    out, lse = torch.zeros_like(q), torch.zeros((32, q.shape[0]), device=DEV)
    a = pg.PagedAttentionArgs((q.data_ptr(), 0, *q.stride()[:2]), (out.data_ptr(), 0, *out.stride()[:2]),
                              pg.Pool.from_buffer_copy(p.packed), lse.data_ptr(), table.data_ptr(), start.data_ptr(), lens.data_ptr(),
                              3, q.shape[0], 600, table.shape[1] * 64, table.shape[1], 32, 0, 0, dim ** -0.5)

    def call(cta, tile):
        torch.cuda.synchronize()
        o = serving.WaitTestOpts(30, cta, tile)
        assert pg.library().splitzip_paged_attention_test(ctypes.byref(a), ws.data_ptr(), ws.numel(), None, ctypes.byref(o)) == sz.OK
        return serving.splitzip_attention_status(ws)

    for cta in (152, 170, 241, 300):
        out.zero_()
        lse.zero_()
        assert call(cta, 1) == sz.ERR_TIMEOUT
        lost = torch.isnan(lse)
        assert 0 < int(lost.sum()) <= 256, "rows of one row tile"
        heads = lost.any(1).nonzero().flatten() // 4
        assert len(heads.unique()) == 1, "rows of one key/value head"
        assert torch.equal(torch.isnan(out), lost.T[..., None].expand_as(out))
        assert torch.equal(lse[~lost], good_lse[~lost]) and torch.equal(out[~lost.T], good[~lost.T])
    assert call(0xFFFFFFFF, 0xFFFFFFFF) == sz.OK
    assert torch.equal(out, good) and torch.equal(lse, good_lse)


@pytest.mark.parametrize("fmt", WIDENED)
@pytest.mark.parametrize("batch,count,tokens", [(9, 600, 4000), (5, 800, 700), (12, 560, 8000)])
def test_ranges_that_overlap_under_widened_caches(batch, count, tokens, fmt):
    """Starts that go back bring more long sequences than the workspace has room for widened: those that it has none for
    are NaN or left out, nothing is written behind the buffers, and ranges in order are right again after it."""
    q, p, table, _, lens = batch_of([count] + [0] * (batch - 1), [tokens] * batch, 8, 2, 64, 16, fmt, seed=batch)
    start = ints([0, count] * (batch // 2 + 1))[: batch + 1]
    size = pg.splitzip_paged_attention_workspace_bytes(q, p, table, count)
    room = torch.zeros(size + (64 << 20), dtype=torch.uint8, device=DEV)
    room[size:] = 0x5A
    out, lse = torch.zeros((count + 1, 8, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((9, count), device=DEV)
    for _ in range(2):
        pg.splitzip_paged_attention(q, p, table, start, lens, out[:count], room[:size], count, lse=lse[:8])
        assert serving.splitzip_attention_status(room[:size]) == sz.OK
    assert bool((room[size:] == 0x5A).all()) and not out[count].any() and not lse[8].any()
    start[2:] = count
    pg.splitzip_paged_attention(q, p, table, start, lens, out[:count], room[:size], count, lse=lse[:8])
    for rows, o, l, tol, ltol in pages_ref.attention(q, p, table, start, lens, table.shape[1] * 16, 0, 0, 0.125):
        close(out[rows], o, tol, "out")
        close(lse[:8][:, rows], l, ltol, "lse")
