"""The operators around the KV cache (norm and rotation, attention, attention
weight, eviction) against their definitions in 64 bits."""
import math

import pytest
import torch

from lossless_bf16_kv_gb300 import serving
from lossless_bf16_kv_gb300 import splitzip as sz
from tests import serving_ref as ref
from tests.gpu_helpers import ensure_library

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPE = {"bf16": torch.bfloat16, "e5m2": torch.float8_e5m2}


@pytest.fixture(autouse=True)
def _built():
    ensure_library()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def make(b, tq, tk, hq, hk, d, fmt="bf16", seed=0):
    """Queries and a cache [b, 2, tk, hk, d] with values of uneven channels."""
    g = gen(seed)
    q = torch.randn((b, tq, hq, d), generator=g, device=DEV).bfloat16()
    kv = torch.randn((b, 2, tk, hk, d), generator=g, device=DEV)
    kv[:, 1] *= torch.exp(torch.randn((hk, d), generator=g, device=DEV))
    return q, kv.to(DTYPE[fmt])


def lens_of(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def attend(q, kv, lens, window=0, sinks=0, scale=None, out=None, ws=None, stream=None):
    out = torch.full_like(q, float("nan")) if out is None else out
    lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), float("nan"), device=DEV)
    ws = serving.alloc_attention_workspace(q, kv[:, 0], window, sinks) if ws is None else ws
    serving.splitzip_attention(q, kv[:, 0], kv[:, 1], out, ws, lens=lens, lse=lse, window=window, sinks=sinks,
                               scale=scale, stream=stream)
    return out, lse


def close(got, want, tol, what=""):
    got = got.double()
    both = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    over = ((got - want).abs() - tol)[both]
    assert over.numel() == 0 or over.max().item() <= 0, \
        f"{what}: {(over > 0).sum().item()} of {over.numel()} past the bound, worst by {over.max().item():.3g}"


def check_attention(q, kv, lens, window=0, sinks=0, scale=None, stream=None):
    b, tq, _, d = q.shape
    full = torch.full((b,), kv.shape[2], dtype=torch.int32, device=DEV) if lens is None else \
        lens.clamp(0, kv.shape[2])
    got, lse = attend(q, kv, lens, window, sinks, scale, stream=stream)
    o, l, tol, ltol = ref.attention(q, kv[:, 0], kv[:, 1], full, window, sinks, d ** -0.5 if scale is None else scale)
    close(got, o, tol, "out")
    close(lse, l, ltol, "lse")


SHAPES = [  # b, q_tokens, kv_tokens, q_heads, kv_heads, dim
    (1, 1, 1, 1, 1, 64), (1, 1, 17, 4, 4, 128), (2, 1, 300, 32, 8, 128), (3, 1, 1000, 8, 1, 64),
    (1, 2, 129, 12, 4, 64), (2, 5, 257, 15, 5, 128), (1, 1, 5000, 40, 8, 128), (1, 4, 64, 64, 1, 128),
    (2, 16, 16, 8, 8, 64), (1, 33, 700, 6, 2, 128), (2, 100, 333, 10, 2, 64), (1, 130, 130, 8, 2, 128),
    (1, 300, 1111, 4, 4, 128), (2, 257, 600, 14, 2, 64), (1, 640, 640, 8, 1, 128), (1, 513, 2000, 5, 5, 64),
]


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("shape", SHAPES)
def test_attention_causal(shape, fmt):
    q, kv = make(*shape, fmt=fmt, seed=sum(shape))
    check_attention(q, kv, None)


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 1), (64, 4), (100, 130), (129, 64), (256, 0), (5000, 3),
                                          (0x80000000, 0)])
@pytest.mark.parametrize("shape", [(2, 1, 900, 8, 2, 128), (1, 3, 700, 12, 3, 64), (2, 300, 900, 8, 2, 128),
                                   (1, 450, 450, 6, 6, 64)])
def test_attention_window_and_sinks(shape, window, sinks, fmt):
    q, kv = make(*shape, fmt=fmt, seed=window % 1000 + sinks)
    check_attention(q, kv, None, window, sinks)


@pytest.mark.parametrize("tq", [1, 4, 40, 200])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 2)])
def test_attention_ragged_lengths_leave_rows_empty(tq, window, sinks):
    """Lengths from zero, shorter than the queries, out of range; a query before
    the sequence's start sees nothing: zero, and -inf."""
    tk = 400
    lens = lens_of([0, 1, tq // 2, tq, 399, 400, 5000, -3])
    q, kv = make(8, tq, tk, 8, 2, 128, seed=tq)
    check_attention(q, kv, lens, window, sinks)
    out, lse = attend(q, kv, lens, window, sinks)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    assert bool((out[7] == 0).all()) and bool((lse[7] == -math.inf).all())


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("tq", [1, 3, 140, 400])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_ignores_what_it_does_not_see(tq, bad, fmt):
    """Slots past the length, outside the window and (for earlier queries) in the
    future hold NaN or infinities in keys and values."""
    tk, window, sinks = 900, 100, 2
    q, kv = make(2, tq, tk, 6, 2, 128, fmt=fmt, seed=tq)
    lens = lens_of([777, 640])
    for i, n in enumerate(lens.tolist()):
        kv[i, :, n:] = bad
        kv[i, :, sinks: max(sinks, n - tq - window - 1)] = bad   # outside every window
        if tq > 1:
            kv[i, 1, n - 1] = bad             # the last slot: seen by the last query only
            kv[i, 1, n - 2, 0, 3] = bad
            kv[i, 1, n - tq + 1 - window, :, 5] = bad   # leaves the window after the first query
    check_attention(q, kv, lens, window, sinks)


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (130, 0), (300, 130), (64, 4), (1, 0)])
@pytest.mark.parametrize("shape", [(1, 3, 129, 24, 3, 64), (2, 1, 255, 64, 1, 128), (1, 16, 257, 16, 2, 64), (2, 42, 700, 6, 2, 128),
                                   (1, 100, 1000, 2, 2, 64), (3, 9, 641, 8, 1, 128), (1, 4, 5000, 40, 2, 64), (1, 128, 384, 3, 3, 128)])
def test_attention_of_up_to_128_rows(shape, window, sinks, fmt):
    """17 to 128 query rows of a key/value head, an odd or even number of tiles of
    128 slots, a first or second one that only some rows see."""
    q, kv = make(*shape, fmt=fmt, seed=shape[2] + window)
    check_attention(q, kv, None, window, sinks)
    b, tq, tk = shape[:3]
    lens = lens_of([min(tk, tq + 100 * i + 3) for i in range(b)])
    kv[0, :, int(lens[0]):] = float("nan")
    check_attention(q, kv, lens, window, sinks)


@pytest.mark.parametrize("scale", [-0.1, 0.0])
@pytest.mark.parametrize("rows", [3, 20, 70, 300])
def test_attention_negative_and_zero_scale_of_many_rows(rows, scale):
    q, kv = make(1, rows, 600, 2, 2, 128, seed=rows)
    check_attention(q, kv, None, 200, 3, scale=scale)


@pytest.mark.parametrize("rows,tokens", [(64, 300), (64, 1000), (300, 700)])
def test_attention_maxima_that_rise(rows, tokens):
    """Keys that grow with the slot: every tile of slots raises the maximum, in one
    half of its slots or in both; and ones that fall, of which none after the first does."""
    q, kv = make(1, rows, tokens, 2, 2, 128, seed=tokens)
    grow = torch.linspace(0.1, 60.0, tokens, device=DEV)
    for size in (grow, grow.flip(0), torch.where(torch.arange(tokens, device=DEV) % 128 < 64, grow, 0.1)):
        k = kv.clone()
        k[:, 0] = (kv[:, 0].float() * size[:, None, None]).bfloat16()
        check_attention(q, k, None, scale=0.05)


@pytest.mark.parametrize("tq", [1, 200])
def test_attention_visible_nan_and_infinity_stay(tq):
    q, kv = make(1, tq, 500, 4, 2, 128, seed=3)
    kv[0, 1, 10, 0, 7] = float("inf")
    kv[0, 1, 20, 1, 9] = float("nan")
    kv[0, 0, 30, 1, 0] = float("nan")     # a key: every row of head 1 that sees it
    out, lse = attend(q, kv, None)
    assert bool((out[:, :, :2, 7] == math.inf).all())
    assert bool(torch.isfinite(out[:, :, :2, :7]).all()) and bool(torch.isnan(out[:, :, 2:]).all())
    assert bool(torch.isnan(lse[:, 2:]).all()) and bool(torch.isfinite(lse[:, :2]).all())


@pytest.mark.parametrize("tq", [1, 6, 260])
def test_attention_strides_and_orders(tq):
    """Heads before tokens, padded rows, one sequence's cache for a whole batch,
    queries as a slice of a fused projection, output into a wider tensor."""
    b, tk, hq, hk, d = 2, 350, 8, 2, 64
    g = gen(5)
    store = torch.randn((b, hk, 2, tk, d + 8), generator=g, device=DEV).bfloat16()
    kv = store.permute(0, 2, 3, 1, 4)[..., :d]
    fused = torch.randn((b, tq, hq + 2 * hk, d), generator=g, device=DEV).bfloat16()
    q = fused[:, :, :hq]
    wide = torch.zeros((b, hq, tq, 2 * d), dtype=torch.bfloat16, device=DEV)
    out = wide[..., d:].transpose(1, 2)
    got, lse = attend(q, kv, None, out=out)
    o, l, tol, ltol = ref.attention(q, kv[:, 0], kv[:, 1], lens_of([tk] * b), 0, 0, d ** -0.5)
    close(got, o, tol, "out")
    close(lse, l, ltol, "lse")
    assert bool((wide[..., :d] == 0).all())
    check_attention(q, kv[:1].expand(b, -1, -1, -1, -1), None)


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("tq", [1, 200])
@pytest.mark.parametrize("size", [1e-3, 30.0, 1e4])
def test_attention_query_magnitudes(size, tq, fmt):
    """Flat and one-hot softmaxes, and rows far from 1 (E5M2 keys scale them)."""
    q, kv = make(1, tq, 300, 4, 2, 128, fmt=fmt, seed=8)
    check_attention((q.float() * size).bfloat16(), kv, None, scale=0.1 / max(1.0, size / 30))


def test_attention_negative_and_zero_scale():
    q, kv = make(2, 20, 200, 4, 2, 64, seed=1)
    for scale in (-0.2, 0.0):
        check_attention(q, kv, None, 50, 1, scale=scale)


@pytest.mark.parametrize("tq", [1, 150])
def test_attention_workspace_is_reused_across_sizes_and_streams(tq):
    """One workspace through calls of other sizes on a side stream: each call
    leaves it as the next needs it; the same call twice gives the same bits."""
    big_q, big_kv = make(1, tq, 6000, 32, 8, 128, seed=2)
    small_q, small_kv = make(3, 1, 900, 6, 3, 64, seed=3)
    ws = torch.zeros(max(sz_ for sz_ in (serving.splitzip_attention_workspace_bytes(big_q, big_kv[:, 0]),
                                         serving.splitzip_attention_workspace_bytes(small_q, small_kv[:, 0]))),
                     dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    with torch.cuda.stream(side):
        for _ in range(3):
            outs.append((attend(big_q, big_kv, None, ws=ws), attend(small_q, small_kv, None, 200, 2, ws=ws)))
    side.synchronize()
    for o in outs[1:]:
        for x, y in zip(o, outs[0]):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert serving.splitzip_attention_status(ws) == sz.OK
    o, l, tol, ltol = ref.attention(big_q, big_kv[:, 0], big_kv[:, 1], lens_of([6000]), 0, 0, 128 ** -0.5)
    close(outs[0][0][0], o, tol)
    o, l, tol, ltol = ref.attention(small_q, small_kv[:, 0], small_kv[:, 1], lens_of([900] * 3), 200, 2, 64 ** -0.5)
    close(outs[0][1][0], o, tol)


def test_attention_offsets_past_32_bits():
    """A cache whose last slots lie more than 2^32 bytes (and 2^31 elements) in;
    the window keeps the reference small."""
    tk, hk, d, window = 2_200_000, 8, 128, 300
    kv = torch.zeros((1, 2, tk, hk, d), dtype=torch.bfloat16, device=DEV)
    g = gen(1)
    kv[:, :, -800:] = torch.randn((1, 2, 800, hk, d), generator=g, device=DEV).bfloat16()
    kv[:, :, :2] = torch.randn((1, 2, 2, hk, d), generator=g, device=DEV).bfloat16()
    near = torch.cat([kv[:, :, :2], kv[:, :, -798:]], dim=2)    # the same slots, close together
    for tq in (1, 120):
        q = torch.randn((1, tq, 16, d), generator=g, device=DEV).bfloat16()
        got, lse = attend(q, kv, None, window, 2)
        o, l, tol, ltol = ref.attention(q, near[:, 0], near[:, 1], lens_of([800]), window, 2, d ** -0.5)
        close(got, o, tol)
        close(lse, l, ltol)
        w = torch.empty((1, hk, tk), device=DEV)
        serving.splitzip_attention_weights(q, kv[:, 0], lse, w, window=window, sinks=2)
        want, wtol = ref.weights(q, near[:, 0], lse, lens_of([800]), window, 2, d ** -0.5)
        close(torch.cat([w[..., :2], w[..., -798:]], -1), want, wtol)
        assert bool((w[..., 2:-798] == 0).all())


def test_attention_replayed_from_a_cuda_graph():
    """The lengths are read on the device: one capture serves a growing cache."""
    q, kv = make(2, 1, 1000, 8, 2, 128, seed=4)
    lens = lens_of([10, 20])
    out, ws = torch.empty_like(q), serving.alloc_attention_workspace(q, kv[:, 0])
    run = lambda: serving.splitzip_attention(q, kv[:, 0], kv[:, 1], out, ws, lens=lens)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for step in ([10, 20], [11, 999], [1000, 1]):
        lens.copy_(lens_of(step))
        graph.replay()
        o, _, tol, _ = ref.attention(q, kv[:, 0], kv[:, 1], lens, 0, 0, 128 ** -0.5)
        close(out, o, tol, str(step))


# -------------------------------------------------------------- weights

@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 3), (128, 200)])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1, 64), (2, 1, 700, 8, 2, 128), (1, 64, 1000, 32, 8, 128),
                                   (2, 77, 333, 15, 5, 64), (1, 600, 600, 8, 2, 128), (1, 200, 900, 64, 1, 64)])
def test_attention_weights(shape, window, sinks, fmt):
    b, tq, tk = shape[:3]
    q, kv = make(*shape, fmt=fmt, seed=sum(shape) + window)
    lens = lens_of([tk, tk * 2 // 3][:b])
    kv[-1, :, lens[-1]:] = float("nan")
    _, lse = attend(q, kv, lens, window, sinks)
    before = torch.rand((b, shape[4], tk), generator=gen(1), device=DEV)
    got = before.clone()
    serving.splitzip_attention_weights(q, kv[:, 0], lse, got, lens=lens, weights_in=got, window=window, sinks=sinks)
    want, tol = ref.weights(q, kv[:, 0].nan_to_num(0.0) if fmt == "bf16" else kv[:, 0].float().nan_to_num(0.0), lse, lens,
                            window, sinks, shape[5] ** -0.5, before)
    close(got, want, tol)
    again = torch.full_like(got, float("nan"))
    serving.splitzip_attention_weights(q, kv[:, 0], lse, again, lens=lens, window=window, sinks=sinks)
    close(again, want - before.double(), tol)
    # Every query that sees something gives away a weight of one per head.
    rows = (lse > -math.inf).sum().item()
    assert abs(again.double().sum().item() - rows) <= 1e-4 * max(1, rows)


def test_attention_weights_of_the_last_queries():
    q, kv = make(2, 300, 500, 8, 2, 128, seed=6)
    lens = lens_of([500, 310])
    _, lse = attend(q, kv, lens)
    last, lse_last = q[:, -32:], lse[:, :, -32:].contiguous()
    w = torch.empty((2, 2, 500), device=DEV)
    serving.splitzip_attention_weights(last, kv[:, 0], lse_last, w, lens=lens)
    want, tol = ref.weights(last, kv[:, 0], lse_last, lens, 0, 0, 128 ** -0.5)
    close(w, want, tol)


# ----------------------------------------------------- norm and rotation

def rope_table(rows, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk,d,rot", [(1, 32, 8, 128, 128), (1, 1, 1, 64, 8), (7, 5, 5, 64, 32), (131, 12, 4, 128, 64),
                                           (1000, 3, 1, 128, 128), (300, 32, 8, 64, 64), (33, 8, 2, 128, 0)])
def test_norm_rope(n, hq, hk, d, rot, interleaved, fmt):
    g = gen(n + rot)
    qkv = (torch.randn((n, hq + 2 * hk, d), generator=g, device=DEV) * 3).bfloat16()
    w = (0.5 + torch.rand((2, d), generator=g, device=DEV)).bfloat16()
    rows = n + 50
    table = rope_table(rows, rot) if rot else None
    pos = torch.randint(0, rows, (n,), generator=g, device=DEV).int()
    slots = torch.randperm(rows, generator=g, device=DEV)[:n]
    kv = torch.full((2, rows, hk, d), 7.0, device=DEV).to(DTYPE[fmt])
    q_out = torch.empty((n, hq, d), dtype=torch.bfloat16, device=DEV)
    serving.splitzip_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], w[0], w[1], pos, table, slots,
                                  q_out, kv[0], kv[1], eps=1e-5, interleaved=interleaved)
    want, tol = ref.norm_rope(qkv[:, :hq], w[0], pos, table, 1e-5, interleaved)
    close(q_out, want, tol + want.abs() * 2.0 ** -8)
    want, tol = ref.norm_rope(qkv[:, hq:hq + hk], w[1], pos, table, 1e-5, interleaved)
    # E5M2: half of 2^-2 of the value, or half a step of the smallest ones.
    tol = tol + (want.abs() * 2.0 ** -8 if fmt == "bf16" else want.abs() * 2.0 ** -3 + 2.0 ** -17)
    close(kv[0].float()[slots], want, tol)
    assert torch.equal(kv[1].float()[slots], qkv[:, hq + hk:].to(DTYPE[fmt]).float())
    rest = torch.ones(rows, dtype=torch.bool, device=DEV)
    rest[slots] = False
    assert bool((kv.float()[:, rest] == 7.0).all())


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk,d,rot", [(2601, 30, 5, 128, 128), (3001, 23, 1, 128, 16), (5003, 30, 7, 64, 32), (2001, 6, 2, 128, 48)])
def test_norm_rope_of_many_tokens(n, hq, hk, d, rot, interleaved, fmt):
    """Heads that are not a whole number of what a group of lanes takes."""
    test_norm_rope(n, hq, hk, d, rot, interleaved, fmt)


def test_norm_rope_batched_cache_dropped_slots_in_place_and_no_weights():
    b, t, hq, hk, d = 3, 40, 4, 2, 64
    g = gen(2)
    n = 9
    q = torch.randn((n, hq, d), generator=g, device=DEV).bfloat16()
    k, v = (torch.randn((n, hk, d), generator=g, device=DEV).bfloat16() for _ in range(2))
    kv = torch.zeros((b, 2, t, hk, d), dtype=torch.bfloat16, device=DEV)
    seq = torch.tensor([0, 0, 1, 2, 2, 2, 1, 0, 1], device=DEV)
    tok = torch.tensor([0, 39, 5, 1, 2, 39, 6, 7, 8], device=DEV)
    slots = seq * 2 * t + tok
    slots[4] = -1
    slots[6] = 10 ** 12
    pos = tok.int()
    pos[8] = 1000                      # past the table
    table = rope_table(64, d)
    keep = q.clone()
    serving.splitzip_qk_norm_rope(q, k, v, None, None, pos, table, slots, q, kv[:, 0], kv[:, 1])
    in_range = pos.clamp_max(63)
    want, tol = ref.norm_rope(keep, None, in_range, table, 1e-6, False)
    close(q[:8], want[:8], (tol + want.abs() * 2.0 ** -8)[:8])
    assert bool(torch.isnan(q[8]).all())
    want, tol = ref.norm_rope(k, None, in_range, table, 1e-6, False)
    count = 0
    for i in range(n):
        if i in (4, 6):
            continue
        got = kv[seq[i], 0, tok[i]]
        if i == 8:
            assert bool(torch.isnan(got).all())
        else:
            close(got, want[i], (tol + want.abs() * 2.0 ** -8)[i])
        assert torch.equal(kv[seq[i], 1, tok[i]], v[i])
        count += 1
    assert int((kv.view(torch.int16) != 0).any(-1).any(-1).sum()) == 2 * count


def test_norm_rope_special_rows():
    """A row of zeros, of the smallest and of the largest values, infinities and
    NaN; E5M2 rounding at its ends (ties to even, overflow to infinity)."""
    d = 64
    q = torch.zeros((6, 1, d), device=DEV)
    q[1] = 1e-30
    q[2] = 3e38
    q[3, 0, 5] = float("inf")
    q[4, 0, 6] = float("nan")
    q[5] = 1.0
    q = q.bfloat16()
    vals = torch.tensor([57344.0, 59392.0, 61184.0, 61440.0, 65536.0, 1e30, -61440.0, 2.0 ** -16, 2.0 ** -17, 1.5 * 2.0 ** -17,
                         3 * 2.0 ** -17, -2.0 ** -18, float("inf"), float("nan"), 1.125, 1.375], device=DEV)
    v = vals.repeat(6, 1, 4).bfloat16()
    kv = torch.zeros((2, 6, 1, d), device=DEV).to(torch.float8_e5m2)
    out = torch.empty_like(q)
    slots = torch.arange(6, device=DEV)
    serving.splitzip_qk_norm_rope(q, q, v, None, None, None, None, slots, out, kv[0], kv[1], eps=0.0 + 1e-6)
    want = v.float().to(torch.float8_e5m2)
    same = (kv[1].view(torch.uint8) == want.view(torch.uint8)) | (torch.isnan(kv[1].float()) & torch.isnan(want.float()))
    assert bool(same.all())
    assert bool((out[0] == 0).all()) and bool((out[1].float().abs() < 1e-20).all())
    assert bool((out[5] == 1).all()) and bool(torch.isnan(out[4]).all())


# ------------------------------------------------------------- eviction

@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("b,t,h,d,budget,first,last", [(1, 1, 1, 64, 1, 0, 0), (2, 100, 3, 64, 10, 0, 0), (1, 1000, 8, 128, 300, 4, 32),
                                                       (3, 777, 2, 128, 40, 20, 20), (2, 5000, 1, 64, 4999, 4, 16),
                                                       (1, 300, 2, 64, 400, 4, 4), (2, 2500, 4, 128, 1, 0, 0)])
def test_evict(b, t, h, d, budget, first, last, fmt):
    g = gen(t + budget)
    kv = torch.randn((b, 2, t, h, d), generator=g, device=DEV).to(DTYPE[fmt])
    w = torch.randn((b, h, t), generator=g, device=DEV)
    w = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.5, (w * 4).round() / 4, w)   # many ties
    lens = lens_of([t, max(0, t // 2), 0][:b])
    check_evict(kv, w, lens, budget, first, last)


def check_evict(kv, w, lens, budget, first, last):
    b, _, t, h, d = kv.shape
    out = torch.full((b, 2, budget, h, d), 3.0, device=DEV).to(kv.dtype)
    index = torch.full((b, h, budget), 99, dtype=torch.int32, device=DEV)
    w_out = torch.full((b, h, budget), float("nan"), device=DEV)
    lens_out = torch.full((b,), 99, dtype=torch.int32, device=DEV)
    serving.splitzip_evict(kv[:, 0], kv[:, 1], w, out[:, 0], out[:, 1], index, lens=lens, weights_out=w_out,
                           lens_out=lens_out, keep_first=first, keep_last=last)
    bits = torch.int16 if kv.dtype == torch.bfloat16 else torch.uint8
    ns = [t] * b if lens is None else [min(max(x, 0), t) for x in lens.tolist()]
    assert lens_out.tolist() == [min(n, budget) for n in ns]
    for i in range(b):
        for j in range(h):
            keep = ref.evict_slots(w[i, j].tolist(), ns[i], budget, first, last)
            assert index[i, j].tolist() == keep + [-1] * (budget - len(keep))
            at = torch.tensor(keep, dtype=torch.long, device=DEV)
            assert torch.equal(out[i, :, :len(keep), j].view(bits), kv[i, :, at, j].view(bits))
            assert bool((out[i, :, len(keep):, j].view(bits) == 0).all())
            assert torch.equal(w_out[i, j, :len(keep)].view(torch.int32), w[i, j, at].view(torch.int32))
            assert bool((w_out[i, j, len(keep):] == 0).all())


def test_evict_special_weights():
    """NaN lowest, infinities at the ends, -0 equal to 0, all equal, subnormals."""
    t = 64
    nan, inf = float("nan"), float("inf")
    rows = [[nan] * t, [0.0] * t, [-0.0, 0.0] * (t // 2), [inf, -inf, nan, 0.0] * (t // 4), [-inf] * 32 + [nan] * 32,
            [1e-42 * (i % 5) for i in range(t)], [float(-i) for i in range(t)]]
    w = torch.tensor(rows, device=DEV)[None]
    kv = torch.randn((1, 2, t, len(rows), 64), generator=gen(0), device=DEV).bfloat16()
    for budget, first, last in ((1, 0, 0), (20, 0, 0), (33, 3, 5), (8, 4, 4), (63, 0, 1)):
        check_evict(kv, w, None, budget, first, last)


def test_evict_long_row_and_strided_views():
    t = 70_001
    g = gen(9)
    store = torch.randn((1, 2, 2, t, 64), generator=g, device=DEV).bfloat16()      # heads before tokens
    check_evict(store.transpose(2, 3), torch.rand((1, 2, t), generator=g, device=DEV), lens_of([t - 1]), 3000, 4, 64)


# ------------------------------------------------------------ refusals

def test_refusals():
    """Nothing is enqueued, the status says why, and the next call is right."""
    b, tq, tk, hq, hk, d = 1, 2, 64, 4, 2, 64
    q, kv = make(b, tq, tk, hq, hk, d)
    out, ws = torch.zeros_like(q), serving.alloc_attention_workspace(q, kv[:, 0])
    good = dict(q=q, k_cache=kv[:, 0], v_cache=kv[:, 1], out=out, workspace=ws)
    odd = torch.zeros((b, tk, hk, d + 1), dtype=torch.bfloat16, device=DEV)[..., :d]           # rows not 16-byte aligned
    shifted = torch.zeros(tq * hq * d + 4, dtype=torch.bfloat16, device=DEV)[4:].view(b, tq, hq, d)
    bad = [dict(q=q.float()), dict(q=q[..., ::2]), dict(k_cache=kv[:, 0].half()), dict(k_cache=odd), dict(q=shifted),
           dict(v_cache=kv[:, 1].to(torch.float8_e5m2)), dict(v_cache=kv[:, 1, :-1]), dict(out=out[:, :, :2]),
           dict(workspace=ws[:16]), dict(workspace=ws[8:]), dict(lens=lens_of([1, 2])), dict(lens=torch.zeros(1, device=DEV)),
           dict(lse=torch.zeros((b, hq, tq + 1), device=DEV)), dict(window=-1), dict(scale=float("nan")),
           dict(q=q[:, :, :3], out=out[:, :, :3]), dict(k_cache=kv[:, 0, :0], v_cache=kv[:, 1, :0])]
    for i, change in enumerate(bad):
        with pytest.raises(sz.SplitZipError) as err:
            serving.splitzip_attention(**{**good, **change})
        assert err.value.status == sz.ERR_INVALID_ARG, i
    with pytest.raises(ValueError):
        serving.splitzip_attention(**{**good, "q": q.cpu()})
    assert bool((out == 0).all())
    w = torch.zeros((b, hk, tk), device=DEV)
    lse = torch.zeros((b, hq, tq), device=DEV)
    for args in ((q, kv[:, 0], None, w), (q, kv[:, 0], lse, w[:, :, :-1]), (q, kv[:, 0], lse[:, :1], w)):
        with pytest.raises(sz.SplitZipError):
            serving.splitzip_attention_weights(*args)
    small = torch.zeros((b, 2, 8, hk, d), dtype=torch.bfloat16, device=DEV)
    index = torch.zeros((b, hk, 8), dtype=torch.int32, device=DEV)
    for kw in (dict(keep_first=5, keep_last=4), dict(keep_first=-1), dict(weights_out=w)):
        with pytest.raises(sz.SplitZipError):
            serving.splitzip_evict(kv[:, 0], kv[:, 1], w, small[:, 0], small[:, 1], index, **kw)
    with pytest.raises(sz.SplitZipError):
        serving.splitzip_evict(kv[:, 0], kv[:, 1], w, small[:, 0], small[:, 1], index.long())
    n = 3
    x = torch.zeros((n, hq, d), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros((n, hk, d), dtype=torch.bfloat16, device=DEV)
    slots, pos, table = torch.arange(n, device=DEV), torch.arange(n, device=DEV).int(), rope_table(n, d)
    fine = [x, y, y, None, None, pos, table, slots, x, kv[0, 0], kv[0, 1]]
    for i, v in ((0, x.float()), (2, y[:2]), (3, torch.zeros(d, device=DEV)), (5, pos.long()), (5, None),
                 (6, rope_table(n, d + 8)), (6, rope_table(n, 12)), (7, pos), (9, kv[0, 0, :, :1]), (10, kv[0, 1].half())):
        with pytest.raises(sz.SplitZipError):
            serving.splitzip_qk_norm_rope(*fine[:i], v, *fine[i + 1:])
    check_attention(q, kv, None)
