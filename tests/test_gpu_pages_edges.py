"""The paged cache's operators where they can go wrong beyond ordinary batches: every power of a quantised
block, values that are not finite, foreign exponent bytes, large batches, pools of other layouts, pages that
sequences share, workspaces that different calls and graphs share."""
import math

import pytest
import torch

from lossless_bf16_kv_gb300 import pages as pg
from lossless_bf16_kv_gb300 import serving
from lossless_bf16_kv_gb300 import splitzip as sz
from tests import pages_ref as ref
from tests.gpu_helpers import ensure_library
from tests.test_gpu_pages import DEV, FORMATS, attend, batch_of, check, close, fill, gen, ints, pool, randn

pytestmark = pytest.mark.gpu
QUANTISED = ["int8", "e2m1"]
#: (new tokens, q_heads, kv_heads, head_dim): single tokens, tiles of rows, more than 1024 and 2048 rows to a head
COUNTS = [([1, 1, 1], 8, 2, 128), ([1, 2, 1], 8, 2, 64), ([30, 1, 90], 8, 2, 128), ([140, 20, 3], 6, 2, 64),
          ([200, 1, 140], 8, 2, 128), ([300, 64, 1], 8, 2, 64), ([0, 0, 260], 8, 2, 128), ([530, 1, 270], 8, 2, 128)]
ids = [f"{'_'.join(map(str, c))}x{h}x{k}x{d}" for c, h, k, d in COUNTS]


@pytest.fixture(autouse=True)
def _built():
    ensure_library()


def compare(found, out, lse):
    for rows, o, l, tol, ltol in found:
        close(out[rows], o, tol, "out")
        close(lse[:, rows], l, ltol, "lse")


def powers(p, g, fmt, values=True):
    """Every power that the store uses, in a pool's values (or keys), largest codes among the codes."""
    rows, exps = (p.v, p.v_exp) if values else (p.k, p.k_exp)
    low, high = ref.GRID[fmt][2:]
    e = torch.randint(low + 127, high + 128, exps.shape, generator=g, device=DEV)
    e[torch.rand(exps.shape, generator=g, device=DEV) < 0.05] = 0
    exps.copy_(e)
    c = torch.randint(0, 256, rows.shape, generator=g, device=DEV)
    rows.copy_((c.clamp_min(1) - 128) if fmt == "int8" else c)


@pytest.mark.parametrize("fmt", QUANTISED)
@pytest.mark.parametrize("counts,heads,kv_heads,dim", COUNTS, ids=ids)
def test_attention_of_values_with_every_power(counts, heads, kv_heads, dim, fmt):
    q, p, table, start, lens = batch_of(counts, [300, 411, 290], heads, kv_heads, dim, 16, fmt, seed=dim)
    powers(p, gen(1), fmt)
    check(q, p, table, start, lens)


@pytest.mark.parametrize("fmt", QUANTISED)
@pytest.mark.parametrize("counts,heads,kv_heads,dim", COUNTS, ids=ids)
def test_attention_of_keys_with_every_power(counts, heads, kv_heads, dim, fmt):
    q, p, table, start, lens = batch_of(counts, [300, 411, 290], heads, kv_heads, dim, 16, fmt, seed=dim)
    powers(p, gen(2), fmt, values=False)
    check(q, p, table, start, lens, scale=2.0 ** -20)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,heads,kv_heads,dim", COUNTS, ids=ids)
def test_attention_of_values_that_are_not_finite(counts, heads, kv_heads, dim, fmt):
    """Seen NaN and infinities are what they make of the sums, in their own channels only."""
    q, p, table, start, lens = batch_of(counts, [300, 411, 290], heads, kv_heads, dim, 16, fmt, seed=dim + 1)
    for b, tokens in enumerate(([0, 290], [17, 200, 409], [1, 100, 289])):
        for i, t in enumerate(tokens):
            page, at, h = table[b, t // 16].long(), t % 16, i % kv_heads
            if p.v_exp is not None:
                p.v_exp[page, at, h, i] = 255
                p.v[page, at, h] = 0
            else:
                rows = p.v.view(torch.uint8) if fmt == "e5m2" else p.v
                bad = torch.tensor([math.nan, math.inf, -math.inf][i], device=DEV).to(p.v.dtype)
                rows[page, at, h, 3 * i + 1] = bad.view(torch.uint8) if fmt == "e5m2" else bad
    # Weights of some size everywhere: infinity times a weight that 16 bits hold as 0 is NaN.
    check(q, p, table, start, lens, scale=0.01)


@pytest.mark.parametrize("fmt", QUANTISED)
@pytest.mark.parametrize("counts,heads,kv_heads,dim", COUNTS, ids=ids)
def test_attention_of_a_key_that_is_NaN(counts, heads, kv_heads, dim, fmt):
    q, p, table, start, lens = batch_of(counts, [300, 411, 290], heads, kv_heads, dim, 16, fmt, seed=dim + 2)
    for b, t in ((0, 299), (1, 5), (2, 280)):
        page = table[b, t // 16].long()
        p.k_exp[page, t % 16, 1, 2] = 255
        p.k[page, t % 16, 1] = 0
    out, lse = attend(q, p, table, start, lens)
    for rows, o, l, tol, ltol in ref.attention(q, p, table, start, lens, table.shape[1] * 16, 0, 0, dim ** -0.5):
        assert bool(l.isnan().any())
        close(out[rows], o, tol, "out")
        close(lse[:, rows], l, ltol, "lse")


@pytest.mark.parametrize("fmt", QUANTISED)
@pytest.mark.parametrize("counts,heads,kv_heads,dim", COUNTS, ids=ids)
def test_attention_of_hidden_slots_with_any_bytes(counts, heads, kv_heads, dim, fmt):
    """Any codes and any exponent bytes in slots that no query sees, in tiles that queries see partly."""
    window, sinks = 70, 3
    q, p, table, start, lens = batch_of(counts, [300, 411, 290], heads, kv_heads, dim, 32, fmt, seed=dim + 3)
    found = ref.attention(q, p, table, start, lens, table.shape[1] * 32, window, sinks, dim ** -0.5)
    g = gen(4)
    seen = torch.zeros((p.pages, 32), dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens.tolist()):
        s = torch.arange(n, device=DEV)
        s = s[(s < sinks) | (s > n - max(counts[b], 1) - window)]
        seen[table[b].long()[s // 32], s % 32] = True
    for t in (p.k, p.v, p.k_exp, p.v_exp):
        any_bytes = torch.randint(0, 256, t.view(torch.uint8).shape, generator=g, device=DEV).to(torch.uint8)
        t.view(torch.uint8).copy_(torch.where(seen[:, :, None, None], t.view(torch.uint8), any_bytes))
    compare(found, *attend(q, p, table, start, lens, window=window, sinks=sinks))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_of_large_batches(dim, fmt):
    """Long sequences behind the 32nd, the last one among them, between single tokens and sequences left out."""
    counts = [1] * 75
    for b, n in ((7, 0), (33, 20), (34, 150), (40, 0), (64, 140), (70, 9), (74, 33)):
        counts[b] = n
    lens = [1 + (37 * b) % 170 for b in range(75)]
    for b in (33, 34, 64, 70, 74):
        lens[b] += counts[b]
    q, p, table, start, lens = batch_of(counts, lens, 8, 2, dim, 16, fmt, seed=dim, pad=2)
    start[43:] += 2                                                 # sequence 42 holds rows of no one's: 3 instead of 1
    check(q, p, table, start, lens)


@pytest.mark.parametrize("fmt", QUANTISED)
def test_attention_shares_work_out_in_a_large_batch(fmt):
    g = gen(6)
    lens = [int(n) for n in torch.randint(0, 1500, (45,), generator=g, device=DEV)]
    lens[37], lens[44] = 4000, 3500
    q, p, table, start, lens = batch_of([1] * 45, lens, 16, 8, 128, 16, fmt, seed=6)
    wide = torch.full((45, 1 << 13), -1, dtype=torch.int32, device=DEV)
    wide[:, : table.shape[1]] = table
    out, lse = attend(q, p, wide, start, lens)
    compare(ref.attention(q, p, table, start, lens, table.shape[1] * 16, 0, 0, 128 ** -0.5), out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,heads,kv_heads,dim", COUNTS, ids=ids)
def test_attention_of_a_pool_that_lies_token_by_token(counts, heads, kv_heads, dim, fmt):
    q, p, table, start, lens = batch_of(counts, [300, 411, 290], heads, kv_heads, dim, 32, fmt, seed=dim + 5)
    flat = pg.Pages(*[None if t is None else t.contiguous() for t in (p.k, p.v, p.k_exp, p.v_exp)])
    assert flat.k.stride(1) > flat.k.stride(2)
    check(q, flat, table, start, lens)
    near = attend(q, p, table, start, lens)
    assert all(torch.equal(x, y) for x, y in zip(near, attend(q, flat, table, start, lens)))


@pytest.mark.parametrize("fmt", FORMATS)
def test_pools_inside_a_larger_tensor(fmt):
    """Keys and values interleaved in one tensor, layers between a pool's pages."""
    g = gen(7)
    base = pool(12, 16, 4, 128, fmt)
    width = base.k.shape[3]
    both = torch.zeros((12, 3, 2, 2, 16, width), dtype=base.k.dtype, device=DEV)   # page, layer, k/v, head, slot
    exps = torch.zeros((12, 3, 2, 16, 2, 4), dtype=torch.uint8, device=DEV)        # page, layer, k/v, slot, head
    args = [both[:, 1, i].transpose(1, 2) for i in range(2)]
    if fmt in QUANTISED:
        args += [exps[:, 1, i] for i in range(2)]
    p = pg.Pages(*args)
    table = torch.randperm(12, generator=g, device=DEV).view(2, 6).int()
    kv = randn(g, 2, 192, 2, 128).bfloat16()
    t = torch.arange(96, device=DEV)
    slots = torch.cat([table[b].long()[t // 16] * 16 + t % 16 for b in range(2)])
    pg.splitzip_pages_store(kv[0], kv[1], slots, p)
    assert not both.view(torch.uint8)[:, [0, 2]].any() and not exps[:, [0, 2]].any()
    q = randn(g, 71, 6, 128).bfloat16()
    check(q, p, table, ints([0, 1, 71]), ints([90, 96]))
    back = torch.zeros((2, 2, 96, 2, 128), dtype=torch.bfloat16, device=DEV)
    pg.splitzip_pages_load(p, table, None, back[0], back[1])
    for i in range(2):
        assert torch.equal(back[i].double().flatten(0, 1), ref.values(*ref.codes(kv[i], fmt), fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", [1024, 65536])
@pytest.mark.parametrize("counts", [[1], [40], [300]])
def test_large_pages_and_a_pool_of_one(counts, size, fmt):
    q, p, table, start, lens = batch_of(counts, [777], 4, 2, 128, size, fmt, seed=size, spare=0)
    assert p.pages == 1
    check(q, p, table, start, lens)
    check(q, p, table, start, lens, kv_tokens=500)
    check(q, p, table, start, lens, window=33, sinks=5)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[1, 1], [5, 70], [300, 1]])
def test_attention_of_pages_that_sequences_share(counts, fmt):
    """The same prefix's pages in two sequences, and the same page at two places of one."""
    q, p, table, start, lens = batch_of(counts, [400, 410], 8, 2, 128, 16, fmt, seed=9)
    table[1, :12] = table[0, :12]
    table[0, 14] = table[0, 3]
    check(q, p, table, start, lens)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,heads,kv_heads,dim", COUNTS, ids=ids)
def test_attention_without_lse(counts, heads, kv_heads, dim, fmt):
    q, p, table, start, lens = batch_of(counts, [300, 411, 290], heads, kv_heads, dim, 16, fmt, seed=10)
    ws = pg.alloc_paged_attention_workspace(q, p, table, max(counts))
    out = torch.empty_like(q)
    pg.splitzip_paged_attention(q, p, table, start, lens, out, ws, max(counts))
    assert torch.equal(out, attend(q, p, table, start, lens)[0])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,heads,kv_heads,dim", COUNTS, ids=ids)
def test_attention_of_queries_of_any_size(counts, heads, kv_heads, dim, fmt):
    """Queries of zeros, of subnormal and tiny values, of large ones next to a small scale; a NaN stays in its row."""
    q, p, table, start, lens = batch_of(counts, [300, 411, 290], heads, kv_heads, dim, 16, fmt, seed=11)
    out, lse = attend(q, p, table, start, lens)
    for factor in (0.0, 2.0 ** -120, 2.0 ** -60):
        check((q.float() * factor).bfloat16(), p, table, start, lens)
    check((q.float() * 2.0 ** 100).bfloat16(), p, table, start, lens, scale=2.0 ** -104)
    bad = q.clone()
    bad[-1, 1, 5] = math.nan
    out2, lse2 = attend(bad, p, table, start, lens)
    assert bool(out2[-1, 1].isnan().all()) and bool(lse2[1, -1].isnan())
    out2[-1, 1], lse2[1, -1] = out[-1, 1], lse[1, -1]
    assert torch.equal(out2, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("group", [17, 64])
def test_attention_of_wide_groups(group, fmt):
    check(*batch_of([1, 1, 3], [300, 411, 290], 2 * group, 2, 128, 16, fmt, seed=group))
    check(*batch_of([1, 0, 20], [30, 411, 290], group, 1, 64, 16, fmt, seed=group))


@pytest.mark.parametrize("fmt", FORMATS)
def test_different_calls_share_a_workspace(fmt):
    """Every kernel's calls, also the strided cache's, in turn on one workspace: each result as on its own."""
    calls = [batch_of(c, [600, 411, 590], h, k, d, 16, fmt, seed=12) for c, h, k, d in COUNTS]
    calls.append(batch_of([1, 1, 1], [9000, 8000, 2], 8, 2, 128, 16, fmt, seed=13))
    odd = batch_of([200, 300, 1], [600, 411, 590], 8, 2, 128, 16, fmt, seed=14)
    if odd[1].v_exp is not None:                                    # leaves NaN behind in the workspace
        odd[1].v_exp.fill_(255)
        odd[1].v.zero_()
    calls.insert(2, odd)
    most = [int((c[3][1:] - c[3][:-1]).max()) for c in calls]
    ws = max((pg.alloc_paged_attention_workspace(c[0], c[1], c[2], m) for c, m in zip(calls, most)), key=len)
    q = randn(gen(15), 2, 1, 8, 128).bfloat16()
    kv = randn(gen(16), 2, 2, 700, 2, 128).bfloat16()
    n = ints([700, 650])
    plain = torch.zeros_like(q)
    own = serving.alloc_attention_workspace(q, kv[0])
    serving.splitzip_attention(q, kv[0], kv[1], plain, own, n)
    assert own.numel() <= ws.numel()
    alone = [attend(*c) for c in calls]
    for _ in range(2):
        for c, want in zip(calls, alone):
            got = attend(*c, ws=ws)
            assert all(torch.equal(x.nan_to_num(9.0), y.nan_to_num(9.0)) for x, y in zip(got, want))
            strided = torch.zeros_like(q)
            serving.splitzip_attention(q, kv[0], kv[1], strided, ws, n)
            assert torch.equal(strided, plain)


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_graphs_share_a_workspace(fmt):
    calls = [batch_of(c, [600, 411, 590], h, k, d, 16, fmt, seed=17) for c, h, k, d in (COUNTS[0], COUNTS[4])]
    calls.append(batch_of([1, 1, 1], [9000, 8000, 2], 8, 2, 128, 16, fmt, seed=18))
    most = [int((c[3][1:] - c[3][:-1]).max()) for c in calls]
    want = [attend(*c) for c in calls]
    ws = max((pg.alloc_paged_attention_workspace(c[0], c[1], c[2], m) for c, m in zip(calls, most)), key=len)
    outs, graphs = [torch.zeros_like(c[0]) for c in calls], []
    for c, m, out in zip(calls, most, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pg.splitzip_paged_attention(*c, out, ws, m)
        graphs.append(graph)
    for i in (0, 1, 2, 1, 0, 2, 2, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i][0])
    assert serving.splitzip_attention_status(ws) == sz.OK


@pytest.mark.parametrize("fmt", FORMATS)
def test_calls_on_two_streams_at_once(fmt):
    """Each with a workspace of its own, on streams that are passed."""
    calls = [batch_of(c, [600, 411, 590], h, k, d, 16, fmt, seed=19) for c, h, k, d in COUNTS]
    want = [attend(*c) for c in calls]
    ws = [pg.alloc_paged_attention_workspace(c[0], c[1], c[2], int((c[3][1:] - c[3][:-1]).max())) for c in calls]
    outs = [torch.zeros_like(c[0]) for c in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for i, c in enumerate(calls):
            pg.splitzip_paged_attention(*c, outs[i], ws[i], max(COUNTS[i][0]), stream=streams[i % 2])
    torch.cuda.synchronize()
    for out, (o, _) in zip(outs, want):
        assert torch.equal(out, o)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_slot_named_twice_touches_no_other(fmt):
    g = gen(20)
    p = pool(4, 16, 2, 128, fmt)
    kv = randn(g, 2, 20, 2, 128).bfloat16()
    slots = torch.arange(20, device=DEV) + 7
    slots[11] = slots[4]
    before = p.k.view(torch.uint8).clone(), p.v.view(torch.uint8).clone()
    pg.splitzip_pages_store(kv[0], kv[1], slots, p)
    once = torch.ones(20, dtype=torch.bool, device=DEV)
    once[4] = once[11] = False
    for i, (rows, exps) in enumerate(((p.k, p.k_exp), (p.v, p.v_exp))):
        c, e = ref.codes(kv[i, once], fmt)
        s = slots[once]
        want = before[i]
        want[s // 16, s % 16] = c.view(torch.uint8)
        got = rows.view(torch.uint8).clone()
        got[slots[4] // 16, slots[4] % 16] = want[slots[4] // 16, slots[4] % 16]
        assert torch.equal(got, want)
        if e is not None:
            assert torch.equal(exps[s // 16, s % 16], e)


@pytest.mark.parametrize("fmt", FORMATS)
def test_load_of_tables_with_a_page_many_times(fmt):
    p = fill(pool(5, 16, 2, 128, fmt), gen(21), fmt)
    table = ints([[3, 3, 3, 1], [3, 0, 3, 3]])
    out = torch.zeros((2, 2, 50, 2, 128), dtype=torch.bfloat16, device=DEV)
    pg.splitzip_pages_load(p, table, None, out[0], out[1])
    for b in range(2):
        for i, x in enumerate("kv"):
            assert torch.equal(out[i, b].double(), ref.sequence(p, table[b], 50, x))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("most", [17, 257, 600, 1500])
def test_attention_of_small_sequences_under_large_bounds(most, fmt):
    """max_q_tokens and the rows of q far above what the sequences bring: every kernel that may run has little or nothing."""
    q, p, table, start, lens = batch_of([1, 3, 0, 2], [300, 411, 290, 5], 8, 2, 128, 16, fmt, seed=most, pad=1500)
    out, lse = check(q, p, table, start, lens, most=most)
    near, near_lse = attend(q[:6], p, table, start, lens)
    close(out[:6].float(), near.double(), 2.0 ** -7 * near.abs().double() + 2.0 ** -6 * near.abs().max().item(), "out")
    assert bool((out[6:] == 7.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_graph_takes_batches_of_any_make_up(fmt):
    """Captured once for 1000 rows; then other ranges, lengths and tables, sequences moving between the kernels."""
    q, p, table, start, lens = batch_of([600, 1, 100, 1], [900, 850, 411, 17], 8, 2, 128, 16, fmt, seed=23, pad=298)
    ws = pg.alloc_paged_attention_workspace(q, p, table, 700)
    out, lse = torch.zeros_like(q), torch.zeros((8, 1000), device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pg.splitzip_paged_attention(q, p, table, start, lens, out, ws, 700, lse=lse)
    full = torch.randperm(p.pages, generator=gen(24), device=DEV)[: table.numel()].view(table.shape).int()
    for starts, n in (([0, 600, 601, 701, 702], [900, 850, 411, 17]), ([0, 1, 2, 3, 4], [912, 1, 0, 500]),
                      ([100, 101, 701, 701, 800], [300, 912, 4, 700]), ([0, 0, 0, 0, 0], [1, 2, 3, 4]),
                      ([3, 260, 517, 774, 1000], [257, 900, 100, 226]), ([0, 800, 1000, 1000, 1000], [900, 900, 900, 900])):
        start.copy_(ints(starts))
        lens.copy_(ints(n))
        table.copy_(full)
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        kept = start.clone()
        if starts[1] - starts[0] > 700:                 # left out
            kept[0] = kept[1]
        mine = torch.zeros(1000, dtype=torch.bool, device=DEV)
        for rows, o, l, tol, ltol in ref.attention(q, p, table, kept, lens, table.shape[1] * 16, 0, 0, 128 ** -0.5):
            close(out[rows], o, tol, "out")
            close(lse[:, rows], l, ltol, "lse")
            mine[rows] = True
        assert bool((out[~mine] == 7.0).all()) and bool((lse[:, ~mine] == 7.0).all())
    assert serving.splitzip_attention_status(ws) == sz.OK


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_at_the_far_end_of_the_lengths(fmt):
    """Positions up to 2^31: a table that names one page again and again.  With a window and sinks, in both kernels;
    and in 8 bits every slot, whose weights are those of the page's, lse more by the log of how often."""
    size, width = 65536, 1 << 15
    n = width * size - 256
    q, p, table, start, _ = batch_of([1], [size], 4, 1, 64, size, fmt, seed=25, spare=0)
    far = torch.zeros((1, width), dtype=torch.int32, device=DEV)
    g = gen(26)
    for count in (1, 3, 40):
        x = randn(g, count, 4, 64).bfloat16()
        window, sinks = 500, 5
        out, lse = attend(x, p, far, ints([0, count]), ints([n]), window=window, sinks=sinks, kv_tokens=n)
        # The same slots in a short cache: the sinks' page in front, the window's end where the far one has it.
        near = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
        for rows, o, l, tol, ltol in ref.attention(x, p, near, ints([0, count]), ints([2 * size - 256]), 2 * size, window,
                                                   sinks, 64 ** -0.5):
            close(out[rows], o, tol, "out")
            close(lse[:, rows], l, ltol, "lse")
    if fmt == "int8":
        n = width * size // 2
        out, lse = attend(q, p, far, ints([0, 1]), ints([n]), kv_tokens=n)
        (rows, o, l, tol, ltol), = ref.attention(q, p, ints([[0]]), ints([0, 1]), ints([size]), size, 0, 0, 64 ** -0.5)
        # A split's sum has up to 2^30 terms in 32 bits, of which a lane's chain has at most 2^30 / 2^13.
        close(out, o, tol + 2.0 ** -7 * o.abs().amax(), "out")
        close(lse, l + math.log(n // size), ltol + 2.0 ** -7, "lse")


@pytest.mark.parametrize("fmt", FORMATS)
def test_keys_and_values_in_one_tensor(fmt):
    q, p, table, start, lens = batch_of([1, 30], [300, 411], 8, 2, 128, 16, fmt, seed=27)
    check(q, pg.Pages(p.k, p.k, p.k_exp, p.k_exp), table, start, lens)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch,tokens", [(10, 4000), (15, 6500)], ids=["pieces", "thirds"])
def test_attention_cuts_the_last_wave(batch, tokens, dim, fmt):
    """Row tiles for a wave of CTAs and some more, which are cut into pieces: full batches, ones that bring fewer row
    tiles than planned, short caches, a window; several calls on one workspace, all alike."""
    q, p, table, start, lens = batch_of([300] * batch, [tokens] * batch, 8, 8, dim, 64, fmt, seed=batch + dim)
    ws = pg.alloc_paged_attention_workspace(q, p, table, 300)
    scale = dim ** -0.5

    def calls(start, lens, window=0, sinks=0):
        out, lse = attend(q, p, table, start, lens, most=300, window=window, sinks=sinks, ws=ws)
        compare(ref.attention(q, p, table, start, lens, table.shape[1] * 64, window, sinks, scale), out, lse)
        for _ in range(3):
            assert torch.equal(attend(q, p, table, start, lens, most=300, window=window, sinks=sinks, ws=ws)[0], out)

    calls(start, lens)
    few = start.clone()
    few[2:] = few[2]                                                # two sequences with new tokens
    calls(few, lens)
    some = start.clone()
    some[4:7] = some[4]                                             # two sequences without, one with too many
    calls_lens = lens.clone()
    calls_lens[0], calls_lens[1], calls_lens[9] = 0, 290, tokens // 2
    out, lse = attend(q, p, table, some, calls_lens, most=300, ws=ws)
    kept = some.clone()
    found = [x for x in ref.attention(q, p, table, kept, calls_lens, table.shape[1] * 64, 0, 0, scale)
             if x[0].stop - x[0].start <= 300]
    compare(found, out, lse)
    assert bool((out[4 * 300: 7 * 300] == 7.0).all())
    calls(start, lens, window=3500, sinks=2)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("batch,count,heads", [(9, 1024, 1), (17, 700, 2), (5, 300, 8), (40, 20, 2), (40, 3, 8)])
def test_ranges_that_overlap_stay_inside_the_buffers(batch, count, heads, fmt):
    """Starts that go back and forth bring more rows than q has, under a bound that has long caches cut."""
    q, p, table, _, lens = batch_of([count] + [0] * (batch - 1), [4000] * batch, heads, heads, 64, 16, fmt, seed=batch)
    start = ints([0, count] * (batch // 2 + 1))[: batch + 1]
    wide = torch.full((batch, 1 << 14), -1, dtype=torch.int32, device=DEV)       # 262144 tokens
    wide[:, : table.shape[1]] = table
    size = pg.splitzip_paged_attention_workspace_bytes(q, p, wide, count)
    assert size
    room = torch.zeros(size + (64 << 20), dtype=torch.uint8, device=DEV)
    room[size:] = 0x5A
    lse = torch.zeros((heads + 1, count), device=DEV)
    out = torch.zeros((count + 1, heads, 64), dtype=torch.bfloat16, device=DEV)
    for _ in range(2):
        pg.splitzip_paged_attention(q, p, wide, start, lens, out[:count], room[:size], count, lse=lse[:heads])
        assert serving.splitzip_attention_status(room[:size]) == sz.OK
    assert bool((room[size:] == 0x5A).all()) and not out[count].any() and not lse[heads].any()
    # The same workspace, ranges in order again.
    start[2:] = count
    check_out, check_lse = torch.zeros_like(out), torch.zeros_like(lse)
    pg.splitzip_paged_attention(q, p, wide, start, lens, check_out[:count], room[:size], count, lse=check_lse[:heads])
    compare(ref.attention(q, p, table, start, lens, table.shape[1] * 16, 0, 0, 0.125), check_out, check_lse[:heads])
