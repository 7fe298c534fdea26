"""The paged cache's operators (store, load, attention) against their definitions in
64 bits."""
import math

import pytest
import torch

from lossless_bf16_kv_gb300 import pages as pg
from lossless_bf16_kv_gb300 import serving
from lossless_bf16_kv_gb300 import splitzip as sz
from tests import pages_ref as ref
from tests.gpu_helpers import ensure_library

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = ["bf16", "e5m2", "int8", "e2m1"]


@pytest.fixture(autouse=True)
def _built():
    ensure_library()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.uint8)


def pool(pages, size, heads, dim, fmt, heads_first=True):
    """A pool of garbage: every byte 0xA5, so that what no call writes is seen."""
    p = pg.alloc_pages(pages, size, heads, dim, fmt)
    if not heads_first:
        rows = [None if t is None else t.contiguous() for t in (p.k, p.v, p.k_exp, p.v_exp)]
        p = pg.Pages(*rows)
    for t in (p.k, p.v, p.k_exp, p.v_exp):
        if t is not None:
            t.view(torch.uint8).fill_(0xA5)
    return p


def fill(p, g, fmt):
    """Keys of uneven length and values of uneven channels in every slot, by the definition."""
    size, heads, dim = p.page_tokens, p.kv_heads, p.head_dim
    for rows, exps, channel in ((p.k, p.k_exp, 0.3), (p.v, p.v_exp, 1.0)):
        x = (randn(g, p.pages, size, heads, dim) * torch.exp(channel * randn(g, heads, dim))).bfloat16()
        c, e = ref.codes(x, fmt)
        rows.view(torch.uint8).copy_(c.view(torch.uint8)) if fmt == "e5m2" else rows.copy_(c)
        if e is not None:
            exps.copy_(e)
    return p


# ------------------------------------------------------------------ store

def special_rows(n, heads, dim, g):
    """Rows with blocks of zeros, infinities, NaN, subnormal and huge values, ties and every magnitude."""
    x = randn(g, n, heads, dim) * torch.exp2(torch.randint(-12, 6, (n, heads, 1), generator=g, device=DEV).float())
    x = x.bfloat16()
    every = torch.arange(0x8000, device=DEV).to(torch.int16).view(torch.bfloat16)   # every magnitude, in order
    flat = x.view(-1)
    flat[: min(flat.numel(), 0x7F80)] = every[: min(flat.numel(), 0x7F80)]
    neg = torch.rand(x.shape, generator=g, device=DEV) < 0.5
    x = torch.where(neg, -x, x)
    block = dim // 4
    x[-1, :, :block] = 0.0
    x[-1, :, 1] = -0.0
    x[-1, 0, block] = math.inf
    x[-1, 0, 2 * block + 3] = -math.inf
    x[-2, :, 3 * block + 1] = math.nan
    x[-3] = 3.0e38
    x[-4] = 1.0e-40
    # Ties of either format: odd eighths next to a largest value that fixes the power.
    x[-5] = (torch.arange(dim, device=DEV) % 32 - 16).bfloat16() * 0.125
    x[-5, :, ::block] = 4.0
    x[-6] = (torch.arange(dim, device=DEV) % 64 - 31.5).bfloat16()
    x[-6, :, ::block] = 64.0
    x[-7, :, ::block] = torch.tensor([127.0, 127.5, 255.0, 7.0], device=DEV).bfloat16()   # at the borders of a power
    return x


@pytest.mark.parametrize("heads_first", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fmt", FORMATS)
def test_store_is_the_definition_bit_for_bit(fmt, dim, heads_first):
    g = gen(dim)
    n, heads, size, pages = 211, 3, 16, 20
    kv = torch.stack([special_rows(n, heads, dim, g), special_rows(n, heads, dim, g).flip(0)], 1)   # slices of one tensor
    p = pool(pages, size, heads, dim, fmt, heads_first)
    before = [None if t is None else t.clone() for t in (p.k, p.v, p.k_exp, p.v_exp)]
    slots = torch.randperm(pages * size, generator=g, device=DEV)[:n]
    slots[3], slots[50], slots[n - 1], slots[n - 2] = -1, pages * size, 1 << 40, -(1 << 62)
    pg.splitzip_pages_store(kv[:, 0], kv[:, 1], slots, p)
    there = ((slots >= 0) & (slots < pages * size)).nonzero().flatten()
    page, at = slots[there] // size, slots[there] % size
    for i in range(2):
        want_rows, want_exps = before[i], before[2 + i]
        rows, exps = ref.codes(kv[there, i], fmt)
        want_rows.view(torch.uint8)[page, at] = rows.view(torch.uint8)
        got = (p.k, p.v)[i]
        got_bits, want_bits = got.view(torch.uint8), want_rows.view(torch.uint8)
        if fmt == "e5m2":   # a NaN has several codes
            nan = torch.isnan(want_rows.float())
            assert torch.equal(nan, torch.isnan(got.float()))
            got_bits, want_bits = got_bits.masked_fill(nan, 0), want_bits.masked_fill(nan, 0)
        differ = (got_bits != want_bits).sum().item()
        assert differ == 0, f"{'kv'[i]}: {differ} bytes of codes"
        if exps is not None:
            want_exps[page, at] = exps
            assert torch.equal((p.k_exp, p.v_exp)[i], want_exps), f"{'kv'[i]}: exponent bytes"


@pytest.mark.parametrize("n,heads", [(0, 4), (1, 1), (1, 8), (7, 5), (65, 2)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_store_then_load_gives_the_values_of_the_codes(fmt, n, heads):
    g = gen(n)
    p = pool(9, 16, heads, 128, fmt)
    k, v = randn(g, n, heads, 128).bfloat16(), (8 * randn(g, n, heads, 128)).bfloat16()
    table = ints([[8, 0, 3, 7, 5]])
    t = torch.arange(n, device=DEV)
    pg.splitzip_pages_store(k, v, table[0].long()[t // 16] * 16 + t % 16, p)
    if not n:
        return
    out = torch.full((2, 1, n, heads, 128), math.nan, dtype=torch.bfloat16, device=DEV)
    pg.splitzip_pages_load(p, table, None, out[0], out[1])
    for x, got in ((k, out[0, 0]), (v, out[1, 0])):
        rows, exps = ref.codes(x, fmt)
        assert torch.equal(got.double(), ref.values(rows, exps, fmt))


# ------------------------------------------------------------------- load

@pytest.mark.parametrize("size", [16, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fmt", FORMATS)
def test_load_widens_every_code_exactly(fmt, dim, size):
    """Random bytes for codes (every code of a format), exponent bytes from all that the store writes."""
    g = gen(size)
    pages, heads, tokens = 30, 3, 300
    p = pool(pages, size, heads, dim, fmt)
    for t in (p.k, p.v):
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.view(torch.uint8).shape, generator=g, device=DEV))
    if p.k_exp is not None:
        low, high = ref.GRID[fmt][2:]
        for t in (p.k_exp, p.v_exp):
            e = torch.randint(low + 127, high + 128, t.shape, generator=g, device=DEV)
            e[torch.rand(t.shape, generator=g, device=DEV) < 0.1] = 0
            e[torch.rand(t.shape, generator=g, device=DEV) < 0.1] = 255
            t.copy_(e)
    width = -(-tokens // size)
    table = torch.randint(0, pages, (6, width), generator=g, device=DEV).int()
    lens = ints([0, 1, 299, 300, 5000, -7])
    table[2, 1], table[3, width - 1] = -1, pages            # pages outside the pool: NaN
    table[1, 1:] = 1 << 30                                  # not needed: not looked at
    out = torch.full((6, 2, tokens, heads, dim), 3.0, dtype=torch.bfloat16, device=DEV)
    pg.splitzip_pages_load(p, table, lens, out[:, 0], out[:, 1])
    for b, n in enumerate(lens.clamp(0, tokens).tolist()):
        for i, x in enumerate("kv"):
            want = ref.sequence(p, table[b], n, x)
            got = out[b, i, :n].double()
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num()), (b, x)
            assert bool((out[b, i, n:] == 3.0).all()), "rows behind the length"


def test_load_of_e5m2_as_it_is():
    g = gen(5)
    p = pool(12, 32, 2, 128, "e5m2")
    for t in (p.k, p.v):
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV))
    table = ints([[11, 3, 4], [0, 1, 2]])
    out = torch.zeros((2, 2, 90, 2, 128), dtype=torch.float8_e5m2, device=DEV)
    pg.splitzip_pages_load(p, table, None, out[0], out[1])
    for i, x in enumerate((p.k, p.v)):
        want = x.view(torch.uint8)[table.long()].flatten(1, 2)[:, :90]
        assert torch.equal(out[i].view(torch.uint8), want)


# -------------------------------------------------------------- attention

def close(got, want, tol, what):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    over = ((got - want).abs() - tol)[torch.isfinite(want)]
    assert over.numel() == 0 or over.max().item() <= 0, \
        f"{what}: {(over > 0).sum().item()} of {over.numel()} past the bound, worst by {over.max().item():.3g}"


def batch_of(counts, lens, heads, kv_heads, dim, size, fmt, seed, pad=0, spare=3):
    """(q, pool, table, q_start, lens): sequences' pages shuffled, entries behind a sequence's last page -1."""
    g = gen(seed)
    width = max(1, max(-(-max(n, 0) // size) for n in lens))
    p = fill(pool(len(lens) * width + spare, size, kv_heads, dim, fmt), g, fmt)
    table = torch.randperm(p.pages, generator=g, device=DEV)[: len(lens) * width].view(-1, width).int()
    for b, n in enumerate(lens):
        table[b, -(-max(n, 0) // size):] = -1
    q = (randn(g, sum(counts) + pad, heads, dim) * (0.5 + torch.rand(dim, generator=g, device=DEV))).bfloat16()
    start = torch.tensor([0] + counts).cumsum(0).int().to(DEV)
    return q, p, table, start, ints(lens)


def attend(q, p, table, start, lens, most=None, window=0, sinks=0, scale=None, kv_tokens=None, ws=None, stream=None):
    most = max(1, int((start[1:] - start[:-1]).max())) if most is None else most
    out = torch.full_like(q, 7.0)
    lse = torch.full((q.shape[1], q.shape[0]), 7.0, device=DEV)
    if ws is None:
        ws = pg.alloc_paged_attention_workspace(q, p, table, most, kv_tokens, window, sinks)
    pg.splitzip_paged_attention(q, p, table, start, lens, out, ws, most, kv_tokens, lse=lse, window=window, sinks=sinks,
                                scale=scale, stream=stream)
    assert serving.splitzip_attention_status(ws) == sz.OK
    return out, lse


def check(q, p, table, start, lens, window=0, sinks=0, scale=None, kv_tokens=None, most=None):
    out, lse = attend(q, p, table, start, lens, most, window, sinks, scale, kv_tokens)
    tokens = table.shape[1] * p.page_tokens if kv_tokens is None else kv_tokens
    mine = torch.zeros(q.shape[0], dtype=torch.bool, device=DEV)
    for rows, o, l, tol, ltol in ref.attention(q, p, table, start, lens, tokens, window, sinks,
                                               q.shape[2] ** -0.5 if scale is None else scale):
        close(out[rows], o, tol, "out")
        close(lse[:, rows], l, ltol, "lse")
        mine[rows] = True
    assert bool((out[~mine] == 7.0).all()) and bool((lse[:, ~mine] == 7.0).all()), "rows that are no sequence's"
    return out, lse


SHAPES = [  # new tokens, lengths, q_heads, kv_heads, head_dim, page_tokens
    ([1], [1], 1, 1, 64, 16), ([1], [17], 4, 4, 128, 16), ([1, 1], [300, 299], 32, 8, 128, 32),
    ([1, 1, 1], [1000, 16, 513], 8, 1, 64, 64), ([2], [129], 12, 4, 64, 16), ([5, 3], [257, 31], 15, 5, 128, 16),
    ([1], [5000], 40, 8, 128, 256), ([4], [64], 64, 1, 128, 64), ([16, 16], [16, 16], 8, 8, 64, 16),
    ([33], [700], 6, 2, 128, 32), ([100, 1], [333, 290], 10, 2, 64, 16), ([130], [130], 8, 2, 128, 128),
    ([300, 7, 1], [1111, 7, 1], 4, 4, 128, 16), ([257, 1, 1, 100], [600, 555, 2, 480], 14, 2, 64, 32),
    ([640], [640], 8, 1, 128, 16), ([1, 513], [2000, 1900], 5, 5, 64, 1024), ([1] * 9, list(range(1, 400, 45)), 8, 2, 128, 16),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{sum(s[0])}of{max(s[1])}x{s[2]}x{s[3]}x{s[4]}p{s[5]}")
def test_attention_causal(shape, fmt):
    check(*batch_of(*shape, fmt, seed=sum(shape[1]) + shape[2], pad=3))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 1), (64, 4), (100, 130), (129, 64), (256, 0), (5000, 3), (0x80000000, 0)])
@pytest.mark.parametrize("shape", [([1, 1], [900, 650], 8, 2, 128, 16), ([3], [700], 12, 3, 64, 64),
                                   ([300, 1], [900, 800], 8, 2, 128, 32), ([450], [450], 6, 6, 64, 16)],
                         ids=["one", "three", "mixed", "prompt"])
def test_attention_window_and_sinks(shape, window, sinks, fmt):
    check(*batch_of(*shape, fmt, seed=window % 1000 + sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("count", [1, 4, 40, 200])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 2)])
def test_attention_ragged_lengths_leave_rows_empty(count, window, sinks, fmt):
    """Lengths of zero, shorter than the new tokens, past the bound, negative; sequences without new tokens."""
    lens = [0, 1, count // 2, count, 399, 400, 5000, -3, 333]
    q, p, table, start, _ = batch_of([count] * 4 + [0] + [count] * 4, [400] * 9, 8, 2, 128, 16, fmt, seed=count)
    out, lse = check(q, p, table, start, ints(lens), window, sinks, kv_tokens=400)
    assert bool((out[:count] == 0).all()) and bool((lse[:, :count] == -math.inf).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("count", [1, 3, 140, 400])
def test_attention_ignores_what_it_does_not_see(count, fmt):
    """Slots past the length, outside the window and in the future hold NaN and infinities; pages that no query
    sees are given away."""
    window, sinks = 100, 2
    q, p, table, start, lens = batch_of([count, count], [777, 640], 6, 2, 128, 16, fmt, seed=count)
    for i, n in enumerate(lens.tolist()):
        slots = torch.arange(table.shape[1] * 16, device=DEV)
        first = n - count - window + 1                     # the first slot of the first query's window
        hidden = (slots >= n) | ((slots >= sinks) & (slots < first))
        late = torch.zeros_like(hidden)
        if count > 1:
            late[n - 1] = True                             # seen by the last query only
        for which, bad in ((hidden, math.nan), (late, math.inf)):
            s = slots[which]
            s = s[table[i].long()[s // 16] >= 0]
            page, at = table[i].long()[s // 16], s % 16
            for rows, exps in ((p.k, p.k_exp), (p.v, p.v_exp)):
                if which is late and rows is p.k:
                    continue
                if exps is not None:
                    exps[page, at, 1:3] = 255
                    rows[page, at] = 0
                else:
                    x = torch.full((len(s), 2, 128), bad, device=DEV).to(rows.dtype)
                    rows.view(torch.uint8)[page, at] = x.view(torch.uint8)
        away = (torch.arange(table.shape[1], device=DEV) * 16 >= max(sinks, 16)) & \
               (torch.arange(table.shape[1], device=DEV) * 16 + 15 < first)
        table[i, away] = ints([-1, 1 << 30])[i]
    # The definition does not look at them either: it gets pages of its own there.
    full = table.clone()
    full[(full < 0) | (full >= p.pages)] = p.pages - 1
    out, lse = attend(q, p, table, start, lens, window=window, sinks=sinks)
    for rows, o, l, tol, ltol in ref.attention(q, p, full, start, lens, table.shape[1] * 16, window, sinks, 128 ** -0.5):
        close(out[rows], o, tol, "out")
        close(lse[:, rows], l, ltol, "lse")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("count", [1, 2, 300])
def test_attention_says_where_a_seen_page_is_outside_the_pool(count, fmt):
    q, p, table, start, lens = batch_of([count] * 3, [500, 400, 450], 8, 2, 64, 32, fmt, seed=count)
    table[1, 2] = p.pages
    out, lse = attend(q, p, table, start, lens)
    rows = slice(count, 2 * count)
    assert bool(out[rows].isnan().all()) and bool(lse[:, rows].isnan().all())
    good = torch.ones(3 * count, dtype=torch.bool, device=DEV)
    good[rows] = False
    assert bool(out[good].isfinite().all()) and bool(lse[:, good].isfinite().all())


def test_attention_leaves_out_sequences_with_bad_ranges():
    q, p, table, start, lens = batch_of([4, 4, 4, 4], [100, 100, 100, 100], 4, 2, 128, 16, "int8", seed=1)
    good, _ = attend(q, p, table, start, lens)
    out, lse = attend(q, p, table, ints([0, 4, 2, 17, 16]), lens, most=4)   # good, backwards, too long, backwards
    assert torch.equal(out[:4], good[:4]) and bool((out[4:] == 7.0).all()) and bool((lse[:, 4:] == 7.0).all())
    out, _ = attend(q, p, table, ints([-4, 4, 8, 16, 1 << 30]), lens, most=4)
    assert torch.equal(out[4:8], good[4:8]) and bool((out[:4] == 7.0).all()) and bool((out[8:] == 7.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [1.0, 0.01])
def test_attention_scales_and_strided_queries(fmt, scale):
    q, p, table, start, lens = batch_of([9, 1, 150], [200, 90, 160], 12, 4, 128, 16, fmt, seed=3)
    qkv = torch.zeros((q.shape[0], 20, 128), dtype=torch.bfloat16, device=DEV)
    qkv[:, 4:16] = q
    check(qkv[:, 4:16], p, table, start, lens, scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_splits_long_caches(fmt):
    """Enough slots for many splits of one sequence, joined through the workspace; twice over the same one."""
    q, p, table, start, lens = batch_of([1], [20011], 4, 1, 128, 16, fmt, seed=11)
    ws = pg.alloc_paged_attention_workspace(q, p, table, 1)
    first, _ = attend(q, p, table, start, lens, ws=ws)
    again, _ = attend(q, p, table, start, lens, ws=ws)
    assert torch.equal(first, again)
    check(q, p, table, start, lens)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("counts", [[8, 8, 5], [130], [3, 300, 1]], ids=["tile", "tiles", "mixed"])
def test_attention_walks_many_tiles_of_slots(counts, dim, fmt):
    """Enough slots that every ring of tiles turns many times; several calls on one workspace, all alike."""
    q, p, table, start, lens = batch_of(counts, [5003, 4800, 4999][: len(counts)], 8, 1, dim, 16, fmt, seed=dim)
    ws = pg.alloc_paged_attention_workspace(q, p, table, max(counts))
    first, _ = check(q, p, table, start, lens)
    for _ in range(10):
        again, _ = attend(q, p, table, start, lens, ws=ws)
        assert torch.equal(first, again)


@pytest.mark.parametrize("fmt", ["e5m2", "int8", "e2m1"])
@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 8, 4), (64, 16, 8), (128, 24, 2)])
def test_attention_shares_work_out_by_length(dim, heads, kv_heads, fmt):
    """A bound on the lengths that is so large that the work is shared out on the GPU: lengths far apart, of zero, a
    sequence left out; several calls on one workspace, all alike."""
    lens = [3000, 1, 17, 0, 2900, 64, 1500, 700]
    q, p, table, start, lens = batch_of([1, 1, 1, 1, 0, 1, 1, 1], lens, heads, kv_heads, dim, 16, fmt, seed=heads)
    wide = torch.full((8, 1 << 14), -1, dtype=torch.int32, device=DEV)       # 262144 tokens
    wide[:, : table.shape[1]] = table
    ws = pg.alloc_paged_attention_workspace(q, p, wide, 1)
    out, lse = attend(q, p, wide, start, lens, ws=ws)
    found = ref.attention(q, p, table, start, lens, table.shape[1] * 16, 0, 0, dim ** -0.5)
    for rows, o, l, tol, ltol in found:
        close(out[rows], o, tol, "out")
        close(lse[:, rows], l, ltol, "lse")
    for _ in range(5):
        assert torch.equal(attend(q, p, wide, start, lens, ws=ws)[0], out)
    lens[0], lens[2] = 20, 2999                 # the same workspace, other lengths
    table[2] = table[0]
    wide[:, : table.shape[1]] = table
    out, lse = attend(q, p, wide, start, lens, ws=ws)
    for rows, o, l, tol, ltol in ref.attention(q, p, table, start, lens, table.shape[1] * 16, 0, 0, dim ** -0.5):
        close(out[rows], o, tol, "out")


def test_attention_of_pages_past_32_bits():
    """A pool of over 4 GiB, the sequence's pages at its end."""
    pages, heads, dim = (1 << 32) // (16 * 8 * 128 * 2) + 40, 8, 128
    p = pg.alloc_pages(pages, 16, heads, dim, "bf16")
    g = gen(2)
    last = pg.Pages(p.k[-40:], p.v[-40:])
    fill(last, g, "bf16")
    table = (pages - 40 + torch.randperm(40, generator=g, device=DEV)[:30].view(2, 15)).int()
    q = randn(g, 150, 16, dim).bfloat16()
    check(q, p, table, ints([0, 1, 150]), ints([237, 200]))
    out = torch.zeros((2, 2, 240, heads, dim), dtype=torch.bfloat16, device=DEV)
    pg.splitzip_pages_load(p, table, None, out[0], out[1])
    assert torch.equal(out[0, 1], last.k[table[1].long() - (pages - 40)].flatten(0, 1))


def test_calls_on_a_stream_and_in_a_graph():
    """Store, attention and load, captured once and replayed on other inputs, slots and lengths."""
    g = gen(8)
    p = pool(40, 16, 2, 128, "int8")
    fill(p, g, "int8")
    q, _, table, start, lens = batch_of([1, 1, 1], [200, 150, 33], 8, 2, 128, 16, "int8", seed=9, pad=1)
    new = randn(g, 3, 2, 2, 128).bfloat16()
    slots = torch.zeros(3, dtype=torch.int64, device=DEV)
    out, back = torch.zeros_like(q), torch.zeros((2, 3, 208, 2, 128), dtype=torch.bfloat16, device=DEV)
    ws = pg.alloc_paged_attention_workspace(q, p, table, 1)

    def step():
        pg.splitzip_pages_store(new[:, 0], new[:, 1], slots, p)
        pg.splitzip_paged_attention(q, p, table, start, lens, out, ws, 1)
        pg.splitzip_pages_load(p, table, lens, back[0], back[1])

    def place():
        t = lens.long() - 1
        slots.copy_(table[torch.arange(3, device=DEV), t // 16].long() * 16 + t % 16)

    place()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in ([200, 150, 33], [7, 144, 16], [1, 2, 208]):
        lens.copy_(ints(n))
        table.copy_(torch.randperm(39, generator=g, device=DEV)[:39].view(3, 13).int())
        new.copy_(randn(g, *new.shape))
        q.copy_(randn(g, *q.shape))
        place()
        graph.replay()
        for rows, o, _, tol, _ in ref.attention(q, p, table, start, lens, 208, 0, 0, 128 ** -0.5):
            close(out[rows], o, tol, "out")
        for b in range(3):
            rows, exps = ref.codes(new[b, 0], "int8")
            assert torch.equal(back[0, b, n[b] - 1].double(), ref.values(rows, exps, "int8"))


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
def test_norm_and_rotation_fill_pages_by_slot(fmt):
    """Pages that lie head by head are a cache with gaps between its sequences for splitzip_qk_norm_rope."""
    g = gen(4)
    heads, dim, size = 2, 128, 16
    p = pg.alloc_pages(9, size, heads, dim, fmt)
    n = 50
    q, k, v = (randn(g, n, h, dim).bfloat16() for h in (4, heads, heads))
    table = ints([[5, 2, 8, 0]])
    t = torch.arange(n, device=DEV)
    slots = table[0].long()[t // size] * (p.k.stride(0) // p.k.stride(1)) + t % size
    serving.splitzip_qk_norm_rope(q, k, v, None, None, None, None, slots, q, p.k, p.v)
    plain = torch.zeros((2, n, heads, dim), dtype=p.k.dtype, device=DEV)
    serving.splitzip_qk_norm_rope(q.clone(), k, v, None, None, None, None, t, torch.empty_like(q), plain[0], plain[1])
    out = torch.zeros((2, 1, n, heads, dim), dtype=p.k.dtype, device=DEV)
    pg.splitzip_pages_load(p, table, None, out[0], out[1])
    assert torch.equal(bits(out[:, 0]), bits(plain))
