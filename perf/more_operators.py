"""The operators of a paged KV cache at the sizes a serving worker meets them, for timing and comparison.

Three operators, one chain over one pool of pages: the store that writes new keys and values to their slots in
BF16, E5M2 or quantised to 8 or 4 bits, the load that reads sequences back out of their pages, and the attention
of a batch's new tokens (single ones, chunks, or both) over their sequences' pages.  `run` is one pass: the
library's calls where `own` is true, else the same operator in elementary torch operations in 32 bits.

Quantised rows: head_dim values in four blocks, each a power of two and 8-bit integers or 4-bit floating-point
numbers (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6).  The power is the smallest one
with which the block's largest magnitude does not round past the largest code.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def _case(name, op, batch, kv_tokens, kv_heads, dim, page, fmt, ragged, **more):
    return dict(name=name, op=op, batch=batch, kv_tokens=kv_tokens, kv_heads=kv_heads, dim=dim, page=page, fmt=fmt,
                ragged=ragged, **more)


def _queries(chunks, q_tokens, q_heads, window=0, sinks=0, pad=0):
    return dict(chunks=chunks, q_tokens=q_tokens, q_heads=q_heads, window=window, sinks=sinks, pad=pad)


def listed():
    return [
        # A sequence's first token, stored and read back: pure latency.
        _case("store_one_token_int8", "store", 1, 1, 8, 128, 16, "int8", False),
        # Prompts of different lengths stored in 4 bits and read back; odd heads, 64 dims.
        _case("store_ragged_e2m1", "store", 13, 333, 5, 64, 16, "e2m1", True),
        # One layer of the 16k prefill, stored in 8 bits and read back.
        _case("store_prompt_16k_int8", "store", 1, 16384, 8, 128, 64, "int8", False),
        # A short odd prefix read back, before it is sent: latency.
        _case("load_short_e2m1", "load", 1, 77, 4, 64, 16, "e2m1", False),
        # A decode batch's quantised caches of one layer read back to be sent.
        _case("load_16x16k_int8", "load", 16, 16384, 8, 128, 64, "int8", True),
        # A single stream's next token over a short odd cache: latency.
        _case("attention_one_token_bf16", "attention", 1, 1001, 8, 128, 16, "bf16", False, **_queries(0, 1, 32)),
        # A decode batch over 8-bit caches of different lengths.
        _case("attention_decode_16x16k_int8", "attention", 16, 16384, 8, 128, 64, "int8", True, **_queries(0, 1, 32)),
        # A decode batch with a window and sinks over 32k caches in 4 bits.
        _case("attention_decode_32k_window_e2m1", "attention", 24, 32768, 8, 128, 32, "e2m1", True,
              **_queries(0, 1, 32, window=4096, sinks=4)),
        # Two chunks of prompts on top of what is cached; three query heads to a key head, 64 dims, odd sizes.
        _case("attention_chunk_509_bf16", "attention", 2, 6001, 4, 64, 16, "bf16", True, **_queries(2, 509, 12)),
        # A mixed batch, padded for a captured graph: one chunk of a prompt and 24 single tokens.
        _case("attention_mixed_1024_int8", "attention", 25, 8192, 8, 128, 32, "int8", True,
              **_queries(1, 1024, 32, pad=8)),
        # A large chunk of a long prompt over an 8-bit cache.
        _case("attention_chunk_2048_int8", "attention", 1, 8192, 8, 128, 64, "int8", False, **_queries(1, 2048, 32)),
        # The last quarter of the 16k prefill.
        _case("attention_chunk_4096_bf16", "attention", 1, 16384, 8, 128, 128, "bf16", False, **_queries(1, 4096, 32)),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "load", "attention", "attention", "attention"])
    fmt = rng.choice(["bf16", "e5m2", "int8", "int8", "e2m1"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    page = rng.choice([16, 16, 32, 64, 128, 256])
    ragged = rng.random() < 0.6
    if op != "attention":
        kv_tokens = _log(rng, 1, 16384)
        batch = _log(rng, 1, max(1, min(64, 2 ** 18 // kv_tokens)))
        if op == "store":
            batch = max(1, min(batch, 16384 // kv_tokens))
        return dict(op=op, batch=batch, kv_tokens=kv_tokens, kv_heads=kv_heads, dim=dim, page=page, fmt=fmt, ragged=ragged)
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 4, 5, 8])
    kv_tokens = _log(rng, 1, 32768)
    kind = rng.choice(["singles", "singles", "chunks", "mixed"])
    batch = _log(rng, 1, max(1, min(32, 2 ** 27 // (kv_tokens * kv_heads * dim))))
    chunks = 0 if kind == "singles" else batch if kind == "chunks" else rng.randrange(0, batch + 1)
    chunks = min(chunks, 4)
    q_tokens = 1
    if chunks:
        most = max(1, min(4096, kv_tokens, 2 ** 30 // (q_heads * kv_tokens * chunks)))   # scores in all
        q_tokens = _log(rng, 1, most)
    windowed = rng.random() < 0.4
    return dict(op=op, batch=batch, kv_tokens=kv_tokens, kv_heads=kv_heads, dim=dim, page=page, fmt=fmt, ragged=ragged,
                chunks=chunks, q_tokens=q_tokens, q_heads=q_heads, window=_log(rng, 16, 8192) if windowed else 0,
                sinks=rng.choice([0, 1, 4, 130]) if windowed else 0, pad=rng.choice([0, 0, 3, 16]))


# ----------------------------------------------------------- quantised rows

#: of a format: its largest code's value, from where on a magnitude in [1, 2) takes the next power, that power's
#: distance to the magnitude's own, and the powers stored
QUANT = {"int8": (127.0, 255 / 128, 6, (-24, 9)), "e2m1": (6.0, 1.75, 2, (-23, 13))}


def _power(k):
    """2^k in 32 bits, k from -126 to 127: exact, which the exponential functions are not."""
    return (k.int() + 127 << 23).view(torch.float32)


def _quantise(x, fmt):
    """(codes, exponent bytes [..., 4]) of rows [..., dim]: int8 [..., dim], or uint8 [..., dim / 2] with the lower
    value in the lower half byte.  An exponent byte e stands for 2^(e - 127); 0 for a block of zeros, 255 for one
    that holds an infinity or a NaN, with codes 0."""
    top, step, away, (low, high) = QUANT[fmt]
    y = x.float().unflatten(-1, (4, -1))
    most = y.abs().amax(-1)
    odd, zero = ~torch.isfinite(most), most == 0
    m, e = torch.frexp(torch.where(odd, 1.0, most))                      # most = m 2^e, m in [0.5, 1)
    power = (e - 1 - away + (2 * m >= step).int()).clamp(low, high)
    z = torch.where(odd[..., None], 0.0, y) * _power(-power)[..., None]
    exps = torch.where(odd, 255, torch.where(zero, 0, power + 127)).to(torch.uint8)
    if fmt == "int8":
        return z.round().clamp(-top, top).to(torch.int8).flatten(-2), exps
    a = z.abs()
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(z)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), exps


def _values(codes, exps, fmt):
    """32-bit values of rows as they lie in pages (an exponent byte is that of a 32-bit number)."""
    if fmt in ("bf16", "e5m2"):
        return codes.float()
    if fmt == "int8":
        z = codes.float()
    else:
        half = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
        z = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)[half]
    scale = torch.where(exps == 255, math.nan, (exps.int() << 23).view(torch.float32))
    return (z.unflatten(-1, (4, -1)) * scale[..., None]).flatten(-2)


# ----------------------------------------------------------------- inputs

DTYPE = {"bf16": torch.bfloat16, "e5m2": torch.float8_e5m2, "int8": torch.int8, "e2m1": torch.uint8}


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _channel_scale(g, heads, dim):
    """Log-normal scales per (head, channel), as KV activations have them."""
    return torch.exp(_randn(g, heads, dim))


def _lens(case, g):
    """Sequence lengths: full, or spread over [kv / 2, kv] with one sequence full."""
    b, kv = case["batch"], case["kv_tokens"]
    if not case["ragged"]:
        return torch.full((b,), kv, dtype=torch.int32, device=DEV)
    lens = torch.randint(max(1, kv // 2), kv + 1, (b,), generator=g, device=DEV, dtype=torch.int32)
    lens[0] = kv
    return lens


def _keys_values(case, g, *shape):
    """Keys after a per-head norm with a learned weight, values with per-channel scales."""
    h, d = case["kv_heads"], case["dim"]
    k = _randn(g, *shape, h, d) * (0.5 + torch.rand(d, generator=g, device=DEV))
    return k, _randn(g, *shape, h, d) * _channel_scale(g, h, d)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    b, h, d, size, fmt = case["batch"], case["kv_heads"], case["dim"], case["page"], case["fmt"]
    s = dict(case=case)
    # The pool, a page's rows head by head, and each sequence's pages in it: shuffled, -1 behind its last one.
    s["lens"] = _lens(case, g)
    width = -(-case["kv_tokens"] // size)
    pages = b * width + b * width // 8
    table = torch.randperm(pages, generator=g, device=DEV)[: b * width].view(b, width)
    last = -(-s["lens"].long() // size)
    s["table"] = torch.where(torch.arange(width, device=DEV) < last[:, None], table, -1).to(torch.int32)
    row = d // 2 if fmt == "e2m1" else d
    turned = lambda *shape, dtype: torch.zeros(shape, dtype=dtype, device=DEV).transpose(1, 2)  # noqa: E731
    for x in "kv":
        s[x] = turned(pages, h, size, row, dtype=DTYPE[fmt])
        s[x + "_exp"] = turned(pages, h, size, 4, dtype=torch.uint8) if fmt in QUANT else None
    if case["op"] == "store":
        starts = torch.cumsum(s["lens"].long(), 0) - s["lens"].long()
        n = int(s["lens"].sum())
        new_k, new_v = _keys_values(case, g, n)
        s["new_kv"] = torch.stack([new_k, new_v], 1).to(torch.bfloat16)       # [n, 2, heads, dim]
        seq = torch.repeat_interleave(torch.arange(b, device=DEV), s["lens"].long())
        at = torch.arange(n, device=DEV) - starts[seq]
        s["slots"] = table[seq, at // size] * size + at % size
    else:
        for x, y in zip("kv", _keys_values(case, g, pages, size)):
            if fmt in QUANT:
                codes, exps = _quantise(y.to(torch.bfloat16), fmt)
                s[x].copy_(codes)
                s[x + "_exp"].copy_(exps)
            else:
                s[x].copy_(y)
    if case["op"] != "attention":
        s["out"] = torch.zeros((b, 2, case["kv_tokens"], h, d), dtype=torch.bfloat16, device=DEV)   # rows past a length stay
        return s
    # New tokens: of the first `chunks` sequences up to q_tokens, of the others one.
    count = torch.ones(b, dtype=torch.int32, device=DEV)
    c, most = case["chunks"], case["q_tokens"]
    if c:
        count[:c] = most - torch.arange(c, device=DEV) * (most // 2) // c if case["ragged"] else most
    s["q_start"] = torch.cat([count.new_zeros(1), count.cumsum(0, dtype=torch.int32)])
    tokens = int(count.sum()) + case["pad"]
    hq = case["q_heads"]
    s["q"] = (_randn(g, tokens, hq, d) * (0.5 + torch.rand(d, generator=g, device=DEV))).to(torch.bfloat16)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros((hq, tokens), device=DEV)
    s["scale"] = d ** -0.5
    return s


# ------------------------------------------------------------- plain forms

def _gather(s, x, seqs):
    """32-bit rows [sequences, slots, heads, dim] of the sequences' pages; pages behind the last are the pool's first."""
    at = s["table"][seqs].long().clamp_min(0)
    exps = s[x + "_exp"]
    rows = s[x][at].flatten(1, 2)
    return _values(rows, None if exps is None else exps[at].flatten(1, 2), s["case"]["fmt"])


def _plain_load(s):
    c, out = s["case"], s["out"]
    there = torch.arange(c["kv_tokens"], device=DEV) < s["lens"][:, None]
    rows = torch.stack([_gather(s, x, slice(None)) for x in "kv"], dim=1)[:, :, : c["kv_tokens"]]
    out.copy_(torch.where(there[:, None, :, None, None], rows, out))
    return {"kv": out}


def _plain_store(s):
    c = s["case"]
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    for i, x in enumerate("kv"):
        new = s["new_kv"][:, i]
        if c["fmt"] in QUANT:
            codes, exps = _quantise(new, c["fmt"])
            s[x][page, at] = codes
            s[x + "_exp"][page, at] = exps
        elif c["fmt"] == "e5m2":
            s[x].view(torch.uint8)[page, at] = new.float().to(torch.float8_e5m2).view(torch.uint8)
        else:
            s[x][page, at] = new
    return _plain_load(s)


def _plain_attend(s, seqs, most):
    """The sequences `seqs` (a slice), each with at most `most` new tokens, as one padded batch."""
    c, q = s["case"], s["q"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    g = hq // hk
    start, end, n = s["q_start"][:-1][seqs].long(), s["q_start"][1:][seqs].long(), s["lens"][seqs].long()
    i = torch.arange(most, device=DEV)
    row = start[:, None] + i                                     # [b, most]: rows of q
    real = row < end[:, None]
    pos = (n - (end - start))[:, None] + i
    qg = (q[row.clamp_max(q.shape[0] - 1)].float() * s["scale"]).unflatten(2, (hk, g)).permute(0, 2, 3, 1, 4)
    b = qg.shape[0]
    sc = torch.matmul(qg.reshape(b, hk, g * most, d), _gather(s, "k", seqs).permute(0, 2, 3, 1)).view(b, hk, g, most, -1)
    slot = torch.arange(sc.shape[-1], device=DEV)
    see = slot <= pos[..., None]
    if c["window"]:
        see &= (slot > pos[..., None] - c["window"]) | (slot < c["sinks"])
    sc.masked_fill_(~see[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True).clamp_min_(torch.finfo(torch.float32).min)
    p = sc.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hk, g * most, -1), _gather(s, "v", seqs).transpose(1, 2)).view(b, hk, g, most, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(b, most, hq, d)
    lse = (top + total.log()).permute(0, 3, 1, 2, 4).reshape(b, most, hq)
    s["out"][row[real]] = o[real].to(torch.bfloat16)
    s["lse"][:, row[real]] = lse[real].T


def _plain_attention(s):
    c = s["case"]
    if c["chunks"]:
        _plain_attend(s, slice(0, c["chunks"]), c["q_tokens"])
    if c["chunks"] < c["batch"]:
        _plain_attend(s, slice(c["chunks"], None), 1)
    return {"out": s["out"], "lse": s["lse"]}


PLAIN = {"store": _plain_store, "load": _plain_load, "attention": _plain_attention}


# ------------------------------------------------------------------ a pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return PLAIN[c["op"]](s)
    from lossless_bf16_kv_gb300 import pages
    if "pages" not in s:     # the pool's handle and, below, the workspace: kept as a program keeps them
        s["pages"] = pages.Pages(s["k"], s["v"], s["k_exp"], s["v_exp"])
    if c["op"] == "attention":
        if "workspace" not in s:
            s["workspace"] = pages.alloc_paged_attention_workspace(s["q"], s["pages"], s["table"], c["q_tokens"], c["kv_tokens"],
                                                                   c["window"], c["sinks"])
        pages.splitzip_paged_attention(s["q"], s["pages"], s["table"], s["q_start"], s["lens"], s["out"], s["workspace"],
                                       c["q_tokens"], c["kv_tokens"], lse=s["lse"], window=c["window"], sinks=c["sinks"],
                                       scale=s["scale"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "store":
        new = s["new_kv"]
        pages.splitzip_pages_store(new[:, 0], new[:, 1], s["slots"], s["pages"])
    # What was stored is read back, as the values it stands for.
    out = s["out"]
    pages.splitzip_pages_load(s["pages"], s["table"], s["lens"], out[:, 0], out[:, 1])
    return {"kv": out}


# ------------------------------------------------------------------- costs

def _row_bytes(case):
    d = case["dim"]
    return {"bf16": 2 * d, "e5m2": d, "int8": d + 4, "e2m1": d // 2 + 4}[case["fmt"]]


def _pairs(case, length, new):
    """Visible (query, slot) pairs and distinct visible slots of one sequence of this length with `new` new tokens."""
    w, snk = case["window"], case["sinks"]
    pairs = 0
    for p in range(max(0, length - new), length):
        pairs += p + 1 if not w or p + 1 <= w else w + min(snk, p + 1 - w)
    seen = length if not w else min(length, max(0, length - max(0, max(0, length - new) - w + 1)) + snk)
    return pairs, seen


def work(case):
    c = case
    mean = 0.75 if c["ragged"] else 1.0      # lengths and new tokens are spread evenly from half to the whole
    length = max(1, int(c["kv_tokens"] * mean))
    row, full = _row_bytes(c), 2 * c["dim"]
    rows = 2 * c["batch"] * length * c["kv_heads"]
    if c["op"] == "load":
        return {"bytes": rows * (row + full), "flops": 0}
    if c["op"] == "store":      # new rows and the pages, each written or read once, and the read back
        return {"bytes": 2 * rows * (row + full), "flops": 0}
    total = {"bytes": 0, "flops": 0}
    for count, new in ((c["chunks"], max(1, int(c["q_tokens"] * mean))), (c["batch"] - c["chunks"], 1)):
        pairs, seen = _pairs(c, length, new)
        total["bytes"] += count * (c["kv_heads"] * seen * 2 * row + c["q_heads"] * new * (2 * full + 4))
        total["flops"] += count * 4 * c["dim"] * c["q_heads"] * pairs
    return total


# ---------------------------------------------------------------- 64 bits

def _two_to(k):
    """2^k in 64 bits, exactly."""
    return (k.long() + 1023 << 52).view(torch.float64)


def _exact_rows(case, x):
    """What rows [..., dim] of BF16 become by the format's definition."""
    fmt = case["fmt"]
    v = x.double()
    if fmt in ("bf16", "e5m2"):
        return v if fmt == "bf16" else x.to(torch.float8_e5m2).double()
    grid = torch.arange(128.0) if fmt == "int8" else torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    grid = grid.double().to(DEV)
    low, high = QUANT[fmt][3]
    beyond = {"int8": 127.5, "e2m1": 7.0}[fmt]       # half way past the largest code: it, too, rounds past it
    blocks = v.reshape(-1, case["dim"] // 4)
    most = blocks.abs().max(1, keepdim=True).values
    power = torch.full_like(most, low)
    for k in range(low, high):
        power = torch.where(most >= beyond * 2.0 ** k, k + 1.0, power)
    power = _two_to(power)
    size = (blocks.abs() / power).clamp_max(grid[-1])
    up = torch.searchsorted(grid, size).clamp(1, len(grid) - 1)
    a, b = grid[up - 1], grid[up]
    even = (up - 1) % 2 == 0
    near = torch.where(size - a < b - size, a, torch.where(size - a > b - size, b, torch.where(even, a, b)))
    return (torch.sign(blocks) * near * power).reshape(v.shape)


def _exact_values(case, codes, exps):
    """Rows of a pool in 64 bits."""
    fmt = case["fmt"]
    if fmt in ("bf16", "e5m2"):
        return codes.double()
    if fmt == "int8":
        z = codes.double()
    else:
        nibble = torch.stack([codes % 16, codes // 16], -1).flatten(-2).int()
        e, m = nibble // 2 % 4, nibble % 2
        z = torch.where(e == 0, m * 0.5, (1 + 0.5 * m.double()) * _two_to(e - 1)) * (1 - 2 * (nibble // 8))
    return z * _two_to(exps.long() - 127).repeat_interleave(case["dim"] // 4, -1)


def exact(case, seed):
    s, c = prepare(case, seed), case
    lens, size = s["lens"].tolist(), c["page"]
    if c["op"] != "attention":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        first = 0
        for b, n in enumerate(lens):
            for i, x in enumerate("kv"):
                if c["op"] == "store":
                    out[b, i, :n] = _exact_rows(c, s["new_kv"][first:first + n, i])
                else:
                    page = s["table"][b, : -(-n // size)].long()
                    exps = s[x + "_exp"]
                    rows = _exact_values(c, s[x][page], None if exps is None else exps[page])
                    out[b, i, :n] = rows.flatten(0, 1)[:n]
            first += n
        return {"kv": out}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    g, start = c["q_heads"] // c["kv_heads"], s["q_start"].tolist()
    for b, n in enumerate(lens):
        page = s["table"][b, : -(-n // size)].long()
        for h in range(c["kv_heads"]):
            k, v = (_exact_values(c, s[x][page, :, h], s[x + "_exp"][page, :, h] if c["fmt"] in QUANT else None).flatten(0, 1)[:n]
                    for x in "kv")
            for i in range(start[b], start[b + 1], 512):
                j = min(start[b + 1], i + 512)
                p = n - start[b + 1] + torch.arange(i, j, device=DEV)[:, None]
                at = torch.arange(n, device=DEV)[None]
                hidden = at > p
                if c["window"]:
                    hidden = hidden | ((at <= p - c["window"]) & (at >= c["sinks"]))
                sc = torch.einsum("rgd,sd->grs", s["q"][i:j, h * g:(h + 1) * g].double(), k) * s["scale"]
                sc[:, hidden] = -math.inf
                total = torch.logsumexp(sc, -1)
                w = torch.exp(sc - torch.where(total > -math.inf, total, 0.0)[..., None])
                out[i:j, h * g:(h + 1) * g] = torch.einsum("grs,sd->rgd", w, v)
                lse[h * g:(h + 1) * g, i:j] = total
    return {"out": out, "lse": lse}
