"""The operators around the KV cache at the sizes a serving worker meets them, for timing and comparison.

Four operators, one chain over one cache: the per-head norm and rotation that fills it, the attention that
reads it, the attention weight its tokens get, and the eviction that thins it before it is sent.  `run` is one
pass: the library's calls where `own` is true, else the same operator in elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BASE = 10000.0     # rotation base
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # A single stream's next token: 48 rows, pure latency.
        dict(name="norm_rope_one_token", op="norm_rope", tokens=1, q_heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, fmt="bf16", rows=16384),
        # A mixed batch of decode and chunk tokens scattered over an FP8 cache; half the dims rotated, pairwise.
        dict(name="norm_rope_ragged_e5m2", op="norm_rope", tokens=777, q_heads=15, kv_heads=5, dim=64,
             rot=32, interleaved=True, fmt="e5m2", rows=4099),
        # One layer of the 16k prefill.
        dict(name="norm_rope_prefill_16k", op="norm_rope", tokens=16384, q_heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, fmt="bf16", rows=16384),
        # A single stream's next token over a short odd cache: latency.
        dict(name="attention_one_token", op="attention", batch=1, q_tokens=1, kv_tokens=1001, q_heads=32,
             kv_heads=8, dim=128, window=0, sinks=0, fmt="bf16", ragged=False),
        # A decode batch over full caches of different lengths.
        dict(name="attention_decode_16x16k", op="attention", batch=16, q_tokens=1, kv_tokens=16384,
             q_heads=32, kv_heads=8, dim=128, window=0, sinks=0, fmt="bf16", ragged=True),
        # A decode batch with a window and sinks over 32k FP8 caches.
        dict(name="attention_decode_32k_window_e5m2", op="attention", batch=24, q_tokens=1, kv_tokens=32768,
             q_heads=32, kv_heads=8, dim=128, window=4096, sinks=4, fmt="e5m2", ragged=True),
        # A chunk of a prompt on top of what is cached; three query heads to a key head, 64 dims, odd sizes.
        dict(name="attention_chunk_509", op="attention", batch=2, q_tokens=509, kv_tokens=6001, q_heads=12,
             kv_heads=4, dim=64, window=0, sinks=0, fmt="bf16", ragged=True),
        # One layer of the 16k prefill with a window and sinks.
        dict(name="attention_prefill_16k", op="attention", batch=1, q_tokens=16384, kv_tokens=16384,
             q_heads=32, kv_heads=8, dim=128, window=4096, sinks=4, fmt="bf16", ragged=False),
        # The prompt's last 64 queries weigh all of its tokens, before eviction.
        dict(name="weights_last_64_of_16k", op="weights", batch=1, q_tokens=64, kv_tokens=16384, q_heads=32,
             kv_heads=8, dim=128, window=0, sinks=0, fmt="bf16", ragged=False),
        # All queries of two prompts weigh their tokens, added to what earlier chunks gave.
        dict(name="weights_prompt_2x3000", op="weights", batch=2, q_tokens=3000, kv_tokens=3500, q_heads=32,
             kv_heads=8, dim=128, window=0, sinks=0, fmt="bf16", ragged=True),
        # One layer of a short prompt, thinned to half.
        dict(name="evict_1_layer_1025", op="evict", batch=1, kv_tokens=1025, kv_heads=8, dim=64, budget=512,
             first=4, last=32, fmt="bf16", ragged=False),
        # The whole 64-layer prefill cache thinned to 2048 tokens before it is sent.
        dict(name="evict_64_layers_16k", op="evict", batch=64, kv_tokens=16384, kv_heads=8, dim=128,
             budget=2048, first=4, last=64, fmt="bf16", ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "attention", "attention", "weights", "evict"])
    dim = rng.choice([64, 128])
    fmt = rng.choice(["bf16", "bf16", "e5m2"])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 8])
    if op == "norm_rope":
        tokens = _log(rng, 1, 16384)
        # an E5M2 cache is compared value by value: kept small
        rows = tokens + rng.randrange(0, 3000) if fmt == "bf16" else min(tokens, 4000) + rng.randrange(0, 500)
        return dict(op=op, tokens=min(tokens, rows), q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.5, fmt=fmt, rows=rows)
    if op == "evict":
        kv_tokens = _log(rng, 64, 32768)
        batch = _log(rng, 1, max(1, min(64, 2 ** 20 // kv_tokens)))
        budget = max(1, int(kv_tokens * rng.uniform(0.05, 0.9)))
        first = min(rng.choice([0, 4]), budget)
        last = min(rng.choice([0, 32, 64]), budget - first)
        return dict(op=op, batch=batch, kv_tokens=kv_tokens, kv_heads=kv_heads, dim=dim, budget=budget,
                    first=first, last=last, fmt="bf16", ragged=rng.random() < 0.5)
    kv_tokens = _log(rng, 16, 32768)
    q_tokens = 1 if op == "attention" and rng.random() < 0.5 else _log(rng, 1, min(kv_tokens, 8192))
    room = 2 ** 31 // (kv_heads * group * q_tokens * kv_tokens)   # scores in all
    room = min(room, 2 ** 28 // (kv_tokens * kv_heads * dim))      # cached values in all
    batch = _log(rng, 1, max(1, min(32, room)))
    if kv_heads * group * q_tokens * kv_tokens > 2 ** 31:
        q_tokens = max(1, 2 ** 31 // (kv_heads * group * kv_tokens))
    windowed = rng.random() < 0.5
    return dict(op=op, batch=batch, q_tokens=q_tokens, kv_tokens=kv_tokens, q_heads=kv_heads * group,
                kv_heads=kv_heads, dim=dim, window=_log(rng, 16, 8192) if windowed else 0,
                sinks=rng.choice([0, 1, 4, 130]) if windowed else 0, fmt=fmt, ragged=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs

def _dtype(fmt):
    return torch.bfloat16 if fmt == "bf16" else torch.float8_e5m2


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _channel_scale(g, heads, dim):
    """Log-normal scales per (head, channel), as KV activations have them."""
    return torch.exp(_randn(g, heads, dim))


def _lens(case, g):
    """Cache lengths: full, or spread over [max(1, kv/2 - q), kv] with one sequence full."""
    b, kv = case["batch"], case["kv_tokens"]
    if not case["ragged"]:
        return torch.full((b,), kv, dtype=torch.int32, device=DEV)
    low = max(1, kv // 2 - case.get("q_tokens", 0) // 4)
    lens = torch.randint(low, kv + 1, (b,), generator=g, device=DEV, dtype=torch.int32)
    lens[0] = kv
    return lens


def _queries_and_cache(case, g):
    """Queries and keys after a per-head norm with a learned weight (rows of about sqrt(dim) length), values with
    per-channel scales; the cache as [batch, 2, tokens, heads, dim]."""
    b, tq, tk, hq, hk, d = (case[k] for k in ("batch", "q_tokens", "kv_tokens", "q_heads", "kv_heads", "dim"))
    w = 0.5 + torch.rand((2, d), generator=g, device=DEV)
    q = (_randn(g, b, tq, hq, d) * w[0]).to(torch.bfloat16)
    kv = torch.empty((b, 2, tk, hk, d), dtype=_dtype(case["fmt"]), device=DEV)
    kv[:, 0] = (_randn(g, b, tk, hk, d) * w[1]).to(kv.dtype)
    kv[:, 1] = (_randn(g, b, tk, hk, d) * _channel_scale(g, hk, d)).to(kv.dtype)
    return q, kv


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case=case)
    if case["op"] == "norm_rope":
        n, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        scale = torch.cat([_channel_scale(g, hq + hk, d), _channel_scale(g, hk, d)])
        s["qkv"] = (_randn(g, n, hq + 2 * hk, d) * scale).to(torch.bfloat16)     # the fused projection's output
        s["q_weight"] = (0.5 + torch.rand(d, generator=g, device=DEV)).to(torch.bfloat16)
        s["k_weight"] = (0.5 + torch.rand(d, generator=g, device=DEV)).to(torch.bfloat16)
        rows = case["rows"]
        in_order = n == rows
        s["positions"] = (torch.arange(n, device=DEV) if in_order else
                          torch.randint(0, rows, (n,), generator=g, device=DEV)).to(torch.int32)
        s["slots"] = torch.arange(n, device=DEV) if in_order else torch.randperm(rows, generator=g, device=DEV)[:n]
        inv = BASE ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        ang = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * inv
        s["table"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()            # [rows, rot]
        s["q_out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device=DEV)
        s["kv"] = torch.zeros((2, rows, hk, d), dtype=_dtype(case["fmt"]), device=DEV)
        return s
    if case["op"] == "evict":
        b, t, h, d = (case[k] for k in ("batch", "kv_tokens", "kv_heads", "dim"))
        s["kv"] = torch.empty((b, 2, t, h, d), dtype=_dtype(case["fmt"]), device=DEV)
        s["kv"].normal_(generator=g)
        w = torch.exp(2.0 * _randn(g, b, h, t))
        s["weights"] = torch.where(torch.rand((b, h, t), generator=g, device=DEV) < 0.25, 0.0, w)  # some never seen
        s["lens"] = _lens(case, g)
        s["kv_out"] = torch.empty((b, 2, case["budget"], h, d), dtype=s["kv"].dtype, device=DEV)
        s["weights_out"] = torch.empty((b, h, case["budget"]), dtype=torch.float32, device=DEV)
        s["index"] = torch.empty((b, h, case["budget"]), dtype=torch.int32, device=DEV)
        s["lens_out"] = torch.empty((b,), dtype=torch.int32, device=DEV)
        return s
    s["q"], s["kv"] = _queries_and_cache(case, g)
    s["lens"] = _lens(case, g)
    s["scale"] = case["dim"] ** -0.5
    b, tq, hq = case["batch"], case["q_tokens"], case["q_heads"]
    if case["op"] == "attention":
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((b, hq, tq), dtype=torch.float32, device=DEV)
    else:
        s["lse"] = torch.logsumexp(_scores(s), dim=-1).reshape(b, hq, tq).contiguous()
        s["before"] = torch.rand((b, case["kv_heads"], case["kv_tokens"]), generator=g, device=DEV)
        s["weights"] = torch.empty_like(s["before"])
    return s


# ------------------------------------------------------------- plain forms

def _visible(case, lens, rows, cols):
    """[batch, rows, cols]: whether the query row sees the slot."""
    pos = (lens.long() - case["q_tokens"])[:, None, None] + rows[None, :, None]
    slot = cols[None, None, :]
    see = slot <= pos
    if case["window"]:
        see &= (slot > pos - case["window"]) | (slot < case["sinks"])
    return see


def _scores(s):
    """Masked scores [batch, kv_heads, group, q, kv] in 32 bits."""
    c, q, kv = s["case"], s["q"], s["kv"]
    b, tq, hq, d = q.shape
    hk = c["kv_heads"]
    qg = (q.float() * s["scale"]).view(b, tq, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    sc = torch.matmul(qg, kv[:, 0].float().permute(0, 2, 3, 1)).view(b, hk, hq // hk, tq, -1)
    see = _visible(c, s["lens"], torch.arange(tq, device=DEV), torch.arange(sc.shape[-1], device=DEV))
    return sc.masked_fill_(~see[:, None, None], -math.inf)


def _plain_norm_rope(s):
    c = s["case"]
    hq, hk, r = c["q_heads"], c["kv_heads"], c["rot"]
    x = s["qkv"][:, :hq + hk].float()
    w = torch.cat([s["q_weight"].expand(hq, -1), s["k_weight"].expand(hk, -1)]).float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    t = s["table"][s["positions"].long()][:, None]
    cos, sin = t[..., : r // 2], t[..., r // 2:]
    if c["interleaved"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = y[..., : r // 2], y[..., r // 2: r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    y = torch.cat([turned, y[..., r:]], dim=-1)
    s["q_out"].copy_(y[:, :hq])
    kv = s["kv"]
    as_bits = kv.view(torch.uint8) if kv.dtype != torch.bfloat16 else kv
    put = lambda z: z.to(kv.dtype).view(as_bits.dtype)  # noqa: E731
    as_bits[0, s["slots"]] = put(y[:, hq:])
    as_bits[1, s["slots"]] = put(s["qkv"][:, hq + hk:].float())
    return {"q": s["q_out"], "kv": kv}


def _plain_attention(s):
    c, kv = s["case"], s["kv"]
    sc = _scores(s)
    top = sc.amax(-1, keepdim=True).clamp_min_(torch.finfo(torch.float32).min)
    p = sc.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    b, hk, g, tq, tk = p.shape
    o = torch.matmul(p.view(b, hk, g * tq, tk), kv[:, 1].float().transpose(1, 2)).view(b, hk, g, tq, -1)
    o = torch.where(total > 0, o / total, 0.0)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(s["out"].shape))
    s["lse"].copy_((top + total.log()).view(b, hk * g, tq))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_weights(s):
    sc = _scores(s)
    b, hk, g, tq, tk = sc.shape
    lse = s["lse"].view(b, hk, g, tq, 1)
    p = sc.sub_(torch.where(lse > -math.inf, lse, 0.0)).exp_()
    torch.add(s["before"], p.sum((2, 3)), out=s["weights"])
    return {"weights": s["weights"]}


def _plain_evict(s):
    c = s["case"]
    b, t, h, budget = c["batch"], c["kv_tokens"], c["kv_heads"], c["budget"]
    slot = torch.arange(t, device=DEV)
    n = s["lens"].long()[:, None, None]
    kept = (slot < c["first"]) | (slot >= n - c["last"])
    rank = torch.where(slot >= n, 2, torch.where(kept, 0, 1)).expand(b, h, t)     # always kept, by weight, absent
    order = torch.sort(s["weights"], dim=-1, descending=True, stable=True).indices
    second = torch.sort(rank.gather(-1, order), dim=-1, stable=True)
    pick = torch.where(second.values[..., :budget] < 2, order.gather(-1, second.indices[..., :budget]), t)
    pick = pick.sort(dim=-1).values
    there = pick < t
    at = pick.clamp_max(t - 1)
    s["index"].copy_(torch.where(there, pick, -1))
    s["weights_out"].copy_(torch.where(there, s["weights"].gather(-1, at), 0.0))
    s["lens_out"].copy_(s["lens"].clamp_max(budget))
    take = at.transpose(1, 2)[:, None, :, :, None].expand(b, 2, budget, h, c["dim"])
    rows = s["kv"].gather(2, take)
    s["kv_out"].copy_(torch.where(there.transpose(1, 2)[:, None, :, :, None], rows, 0.0))
    return {"kv": s["kv_out"], "weights": s["weights_out"], "index": s["index"], "lens": s["lens_out"]}


PLAIN = {"norm_rope": _plain_norm_rope, "attention": _plain_attention, "weights": _plain_weights,
         "evict": _plain_evict}


# ------------------------------------------------------------------ a pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return PLAIN[c["op"]](s)
    from lossless_bf16_kv_gb300 import serving
    if c["op"] == "norm_rope":
        hq, hk, qkv, kv = c["q_heads"], c["kv_heads"], s["qkv"], s["kv"]
        serving.splitzip_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], s["q_weight"], s["k_weight"],
                                      s["positions"], s["table"], s["slots"], s["q_out"], kv[0], kv[1], eps=EPS,
                                      interleaved=c["interleaved"])
        return {"q": s["q_out"], "kv": kv}
    if c["op"] == "evict":
        kv, out = s["kv"], s["kv_out"]
        serving.splitzip_evict(kv[:, 0], kv[:, 1], s["weights"], out[:, 0], out[:, 1], s["index"], lens=s["lens"],
                               weights_out=s["weights_out"], lens_out=s["lens_out"], keep_first=c["first"],
                               keep_last=c["last"])
        return {"kv": out, "weights": s["weights_out"], "index": s["index"], "lens": s["lens_out"]}
    kv = s["kv"]
    if c["op"] == "attention":
        if "workspace" not in s:     # kept for the sizes, as a program keeps it
            s["workspace"] = serving.alloc_attention_workspace(s["q"], kv[:, 0], c["window"], c["sinks"])
        serving.splitzip_attention(s["q"], kv[:, 0], kv[:, 1], s["out"], s["workspace"], lens=s["lens"], lse=s["lse"],
                                   window=c["window"], sinks=c["sinks"], scale=s["scale"])
        return {"out": s["out"], "lse": s["lse"]}
    serving.splitzip_attention_weights(s["q"], kv[:, 0], s["lse"], s["weights"], lens=s["lens"],
                                       weights_in=s["before"], window=c["window"], sinks=c["sinks"], scale=s["scale"])
    return {"weights": s["weights"]}


# ------------------------------------------------------------------- costs

def _pairs(case, length):
    """Visible (query, slot) pairs and distinct visible slots of one sequence of this length."""
    tq, w, snk = case["q_tokens"], case["window"], case["sinks"]
    p0 = length - tq
    pairs = 0
    for p in range(max(0, p0), length):
        pairs += p + 1 if not w or p + 1 <= w else w + min(snk, p + 1 - w)
    seen = length if not w else min(length, max(0, length - max(0, max(0, p0) - w + 1)) + snk)
    return pairs, seen


def work(case):
    c = case
    e = 2 if c.get("fmt") == "bf16" else 1
    if c["op"] == "norm_rope":
        row = c["dim"] * (c["q_heads"] * 4 + c["kv_heads"] * (4 + 2 * e))
        return {"bytes": c["tokens"] * (row + 4 * c["rot"] + 12) + 4 * c["dim"],
                "flops": c["tokens"] * c["dim"] * (c["q_heads"] + c["kv_heads"]) * 8}
    # ragged lengths are spread evenly from about half the cache to the whole of it
    mean = 0.75 if c["ragged"] else 1.0
    length = max(1, int(c["kv_tokens"] * mean))
    if c["op"] == "evict":
        kept = min(c["budget"], length)
        return {"bytes": c["batch"] * c["kv_heads"] * (4 * length + kept * (4 * c["dim"] * e + 8)), "flops": 0}
    pairs, seen = _pairs(c, length)
    rows = c["batch"] * c["q_heads"] * c["q_tokens"]
    if c["op"] == "attention":
        return {"bytes": c["batch"] * c["kv_heads"] * seen * 2 * c["dim"] * e + rows * (4 * c["dim"] + 4),
                "flops": 4 * c["dim"] * c["batch"] * c["q_heads"] * pairs}
    return {"bytes": c["batch"] * c["kv_heads"] * (seen * c["dim"] * e + 8 * c["kv_tokens"]) + rows * (2 * c["dim"] + 4),
            "flops": 2 * c["dim"] * c["batch"] * c["q_heads"] * pairs}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm_rope":
        return _exact_norm_rope(s)
    if c["op"] == "evict":
        return _exact_evict(s)
    return _exact_attention(s) if c["op"] == "attention" else _exact_weights(s)


def _exact_norm_rope(s):
    c, r = s["case"], s["case"]["rot"]
    hq, hk = c["q_heads"], c["kv_heads"]
    x = s["qkv"].double()
    n = x.shape[0]
    out = torch.empty((n, hq + hk, c["dim"]), dtype=torch.float64, device=DEV)
    angle = torch.complex(*(s["table"].double()[s["positions"].long()].chunk(2, dim=1)))     # cos + i sin
    for h in range(hq + hk):
        v = x[:, h]
        v = v / torch.sqrt((v * v).sum(1, keepdim=True) / c["dim"] + EPS)
        v = v * (s["q_weight"] if h < hq else s["k_weight"]).double()
        if c["interleaved"]:
            z = torch.view_as_complex(v[:, :r].reshape(n, r // 2, 2).contiguous()) * angle
            out[:, h, :r] = torch.view_as_real(z).reshape(n, r)
        else:
            z = torch.complex(v[:, : r // 2].contiguous(), v[:, r // 2: r].contiguous()) * angle
            out[:, h, : r // 2], out[:, h, r // 2: r] = z.real, z.imag
        out[:, h, r:] = v[:, r:]
    kv = torch.zeros((2, c["rows"], hk, c["dim"]), dtype=torch.float64, device=DEV)
    kv[0, s["slots"]] = out[:, hq:]
    kv[1, s["slots"]] = x[:, hq + hk:]
    return {"q": out[:, :hq], "kv": kv}


def _blocks(s):
    """(sequence, kv head, first row, last row + 1, first slot, masked scores [group, rows, slots]) in 64 bits, by blocks of rows."""
    c = s["case"]
    hk, g, tq, d = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["q_tokens"], c["dim"]
    for b in range(c["batch"]):
        n = int(s["lens"][b])
        for h in range(hk):
            k = s["kv"][b, 0, :n, h].double()
            for i in range(0, tq, 1024):
                j = min(tq, i + 1024)
                q = s["q"][b, i:j, h * g:(h + 1) * g].double().transpose(0, 1)
                lo = 0
                if c["window"] and n - tq + i - c["window"] >= c["sinks"]:
                    lo = max(0, n - tq + i - c["window"])
                at = torch.cat([torch.arange(min(c["sinks"], lo), device=DEV), torch.arange(lo, n, device=DEV)])
                p = torch.arange(n - tq + i, n - tq + j, device=DEV)[:, None]
                hidden = at[None] > p
                if c["window"]:
                    hidden |= (at[None] <= p - c["window"]) & (at[None] >= c["sinks"])
                sc = torch.einsum("grd,sd->grs", q, k[at]) * s["scale"]
                sc[:, hidden] = -math.inf
                yield b, h, i, j, at, sc


def _exact_attention(s):
    c = s["case"]
    g = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    for b, h, i, j, at, sc in _blocks(s):
        l = torch.logsumexp(sc, dim=-1)
        p = torch.exp(sc - torch.where(l > -math.inf, l, 0.0)[..., None])
        out[b, i:j, h * g:(h + 1) * g] = torch.einsum("grs,sd->rgd", p, s["kv"][b, 1, at, h].double())
        lse[b, h * g:(h + 1) * g, i:j] = l
    return {"out": out, "lse": lse}


def _exact_weights(s):
    c = s["case"]
    g = c["q_heads"] // c["kv_heads"]
    w = s["before"].double()
    for b, h, i, j, at, sc in _blocks(s):
        l = s["lse"][b, h * g:(h + 1) * g, i:j].double()
        w[b, h, at] += torch.exp(sc - torch.where(l > -math.inf, l, 0.0)[..., None]).sum((0, 1))
    return {"weights": w}


def _exact_evict(s):
    c = s["case"]
    b, t, h, budget = c["batch"], c["kv_tokens"], c["kv_heads"], c["budget"]
    weights, lens = s["weights"].double(), s["lens"].tolist()
    kv = torch.zeros(s["kv_out"].shape, dtype=torch.float64, device=DEV)
    wout = torch.zeros((b, h, budget), dtype=torch.float64, device=DEV)
    index = torch.full((b, h, budget), -1, dtype=torch.int32, device=DEV)
    for i, n in enumerate(lens):
        m = min(n, budget)
        key = weights[i, :, :n].clone()
        if n > budget:
            key[:, : c["first"]] = math.inf
            key[:, n - c["last"]:] = math.inf
            # by weight, then by slot: a slot is kept if fewer than m slots come before it
            low = key.sort(dim=1).values[:, n - m, None]
            over = (key > low).sum(1, keepdim=True)
            equal = key == low
            keep = (key > low) | (equal & (equal.cumsum(1) <= m - over))
            at = keep.nonzero()[:, 1].view(h, m)
        else:
            at = torch.arange(n, device=DEV).expand(h, n)
        index[i, :, :m] = at
        wout[i, :, :m] = weights[i].gather(1, at)
        heads = torch.arange(h, device=DEV)[None]
        kv[i, 0, :m] = s["kv"][i, 0][at.T, heads].double()
        kv[i, 1, :m] = s["kv"][i, 1][at.T, heads].double()
    return {"kv": kv, "weights": wout, "index": index, "lens": s["lens"].clamp_max(budget)}
