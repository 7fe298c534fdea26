"""A prompt's KV cache from prefill to decode, with every operator of this package.

    python -m lossless_bf16_kv_gb300.handoff [--layers 4] [--tokens 2048] [--budget 512] [--fmt bf16|e5m2]
        [--pages bf16|e5m2|int8|e2m1] ...

The prefill worker takes a prompt through the attention part of each layer
(``splitzip_qk_norm_rope`` writes the cache, ``splitzip_attention`` reads it
with a sliding window and sinks, ``splitzip_attention_weights`` weighs its
tokens by the last queries), thins all layers at once (``splitzip_evict``) and
packs what is left for the host link with the lossless codec
(``encode_to_host``, a codebook per layer).  The decode worker unpacks it
(``splitzip_decode_from_host``), appends its own tokens and attends over them, or
(``--pages``) keeps the cache in pages of another format (``splitzip_pages_store``,
``splitzip_paged_attention``).

Projections are random matrices and the prompt random vectors: nothing here is
a trained model.  The cache that arrives is bit for bit the one that was sent.
"""
from __future__ import annotations

import argparse
import math
from dataclasses import dataclass

import torch

from . import pages as paged
from . import serving
from . import splitzip as sz


@dataclass
class Shape:
    layers: int = 4
    tokens: int = 2048
    q_heads: int = 32
    kv_heads: int = 8
    dim: int = 128
    window: int = 1024
    sinks: int = 4
    budget: int = 512      # cached tokens a layer and head keeps at most
    observe: int = 64      # last queries whose attention decides
    steps: int = 8         # tokens decoded
    fmt: str = "bf16"
    seed: int = 0
    pages: str = ""        # the decode worker's pages: bf16, e5m2, int8 or e2m1; "": it keeps the cache as it came
    page_tokens: int = 16

    @property
    def dtype(self) -> torch.dtype:
        return torch.bfloat16 if self.fmt == "bf16" else torch.float8_e5m2

    @property
    def kept(self) -> int:
        """Cached tokens a layer and head keeps: a prompt shorter than the budget keeps all of its own."""
        return min(self.budget, self.tokens)


class Layers:
    """Random projections and norm weights of every layer, and the rotation table."""

    def __init__(self, s: Shape, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(s.seed)
        self.s, self.device = s, device
        hidden = s.q_heads * s.dim
        heads = s.q_heads + 2 * s.kv_heads

        def draw(*shape, scale):
            return (torch.randn(shape, generator=g, device=device) * scale).bfloat16()
        self.qkv = [draw(hidden, heads * s.dim, scale=hidden ** -0.5) for _ in range(s.layers)]
        self.out = [draw(hidden, hidden, scale=hidden ** -0.5) for _ in range(s.layers)]
        self.norm = [(0.5 + torch.rand((2, s.dim), generator=g, device=device)).bfloat16() for _ in range(s.layers)]
        inv = 10000.0 ** (-torch.arange(0, s.dim, 2, device=device, dtype=torch.float64) / s.dim)
        ang = torch.arange(s.tokens + s.steps, device=device, dtype=torch.float64)[:, None] * inv
        self.table = torch.cat([ang.cos(), ang.sin()], dim=1).float()
        self.prompt = draw(s.tokens, hidden, scale=1.0)
        self.new = draw(s.steps, hidden, scale=1.0)

    def project(self, layer: int, x: torch.Tensor):
        """Queries, keys and values [n, heads, dim] of hidden states [n, hidden]: slices of one product."""
        s = self.s
        qkv = (x @ self.qkv[layer]).view(x.shape[0], s.q_heads + 2 * s.kv_heads, s.dim)
        return qkv[:, :s.q_heads], qkv[:, s.q_heads:s.q_heads + s.kv_heads], qkv[:, s.q_heads + s.kv_heads:]

    def mix(self, layer: int, x: torch.Tensor, attended: torch.Tensor) -> torch.Tensor:
        return x + attended.reshape(x.shape[0], -1) @ self.out[layer]


def prefill(m: Layers):
    """(cache [layers, 2, tokens, kv_heads, dim], attention weights [layers, kv_heads, tokens])."""
    s, dev = m.s, m.device
    kv = torch.empty((s.layers, 2, s.tokens, s.kv_heads, s.dim), dtype=s.dtype, device=dev)
    weights = torch.empty((s.layers, s.kv_heads, s.tokens), device=dev)
    slots = torch.arange(s.tokens, device=dev)
    positions = slots.int()
    q = torch.empty((1, s.tokens, s.q_heads, s.dim), dtype=torch.bfloat16, device=dev)
    out, lse = torch.empty_like(q), torch.empty((1, s.q_heads, s.tokens), device=dev)
    workspace = serving.alloc_attention_workspace(q, kv[:1, 0], s.window, s.sinks)
    watch = s.tokens - min(s.observe, s.tokens)     # the first of the last queries
    x = m.prompt
    for layer in range(s.layers):
        qr, kr, vr = m.project(layer, x)
        k, v = kv[layer:layer + 1, 0], kv[layer:layer + 1, 1]
        serving.splitzip_qk_norm_rope(qr, kr, vr, m.norm[layer][0], m.norm[layer][1], positions, m.table, slots, q[0], k, v)
        serving.splitzip_attention(q, k, v, out, workspace, lse=lse, window=s.window, sinks=s.sinks)
        serving.splitzip_attention_weights(q[:, watch:], k, lse[:, :, watch:].contiguous(), weights[layer:layer + 1],
                                           window=s.window, sinks=s.sinks)
        x = m.mix(layer, x, out[0])
    return kv, weights


def thin(s: Shape, kv: torch.Tensor, weights: torch.Tensor):
    """(thinned cache, kept slots [layers, kv_heads, kept]): all layers in one call, as its batch."""
    small = torch.empty((s.layers, 2, s.kept, s.kv_heads, s.dim), dtype=kv.dtype, device=kv.device)
    index = torch.empty((s.layers, s.kv_heads, s.kept), dtype=torch.int32, device=kv.device)
    serving.splitzip_evict(kv[:, 0], kv[:, 1], weights, small[:, 0], small[:, 1], index, keep_first=min(s.sinks, s.kept),
                           keep_last=min(s.observe, s.kept - min(s.sinks, s.kept)))
    return small, index


def send(s: Shape, kv: torch.Tensor):
    """(host payload, its bytes, the cache unpacked from it): through host memory, a codebook per layer."""
    layer = kv[0].numel()
    chunk = math.gcd(layer, 1024)    # a layer is a whole number of chunks
    scratch = sz.alloc_transfer_scratch(layer, chunk, s.fmt)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()     # the transfer runs on streams of its own
    payload, nbytes = sz.encode_to_host(kv.reshape(-1), chunk, None, layer, scratch, streams, s.fmt)
    there = torch.empty_like(kv)
    sz.splitzip_decode_from_host(payload, nbytes, there.reshape(-1), scratch, streams)
    return payload, nbytes, there


def decode(m: Layers, thinned: torch.Tensor):
    """Attention outputs [steps, layers, q_heads, dim] of the new tokens over the thinned cache and themselves,
    their queries likewise, and the cache with the new tokens appended."""
    s, dev = m.s, m.device
    kv = torch.empty((s.layers, 2, s.kept + s.steps, s.kv_heads, s.dim), dtype=thinned.dtype, device=dev)
    kv[:, :, :s.kept] = thinned
    queries = torch.empty((s.steps, s.layers, s.q_heads, s.dim), dtype=torch.bfloat16, device=dev)
    outs = torch.empty_like(queries)
    workspace = serving.alloc_attention_workspace(queries[:1, :1], kv[:1, 0])
    lens = torch.full((1,), s.kept, dtype=torch.int32, device=dev)
    for step in range(s.steps):
        position = torch.full((1,), s.tokens + step, dtype=torch.int32, device=dev)   # in the whole text
        slot = torch.full((1,), s.kept + step, dtype=torch.int64, device=dev)       # in the thinned cache
        lens += 1
        x = m.new[step:step + 1]
        for layer in range(s.layers):
            qr, kr, vr = m.project(layer, x)
            k, v = kv[layer:layer + 1, 0], kv[layer:layer + 1, 1]
            q, out = queries[step:step + 1, layer:layer + 1], outs[step:step + 1, layer:layer + 1]   # [1, 1, q_heads, dim]
            serving.splitzip_qk_norm_rope(qr, kr, vr, m.norm[layer][0], m.norm[layer][1], position, m.table, slot, q[0], k, v)
            serving.splitzip_attention(q, k, v, out, workspace, lens=lens)
            x = m.mix(layer, x, out[0])
    return outs, queries, kv


def decode_paged(m: Layers, thinned: torch.Tensor):
    """As ``decode``, over pages: outputs and queries of the new tokens, the pool and its table [layers, pages]."""
    s, dev = m.s, m.device
    width = -(-(s.kept + s.steps) // s.page_tokens)
    pool = paged.alloc_pages(s.layers * width, s.page_tokens, s.kv_heads, s.dim, s.pages, dev)
    table = torch.arange(s.layers * width, dtype=torch.int32, device=dev).view(s.layers, width)

    def slots(layer: int, t: torch.Tensor) -> torch.Tensor:
        return table[layer, t // s.page_tokens].long() * s.page_tokens + t % s.page_tokens
    here = torch.arange(s.kept, device=dev)
    for layer in range(s.layers):
        k, v = thinned[layer].bfloat16()
        paged.splitzip_pages_store(k, v, slots(layer, here), pool)
    queries = torch.empty((s.steps, s.layers, s.q_heads, s.dim), dtype=torch.bfloat16, device=dev)
    outs = torch.empty_like(queries)
    new = torch.empty((2, 1, s.kv_heads, s.dim), dtype=torch.bfloat16, device=dev)     # a token's keys and values
    first = torch.zeros(1, dtype=torch.int64, device=dev)
    start = torch.arange(2, dtype=torch.int32, device=dev)
    lens = torch.full((1,), s.kept, dtype=torch.int32, device=dev)
    workspace = paged.alloc_paged_attention_workspace(queries[0, :1], pool, table[:1], 1)
    for step in range(s.steps):
        position = torch.full((1,), s.tokens + step, dtype=torch.int32, device=dev)
        lens += 1
        x = m.new[step:step + 1]
        for layer in range(s.layers):
            qr, kr, vr = m.project(layer, x)
            q, out = queries[step, layer:layer + 1], outs[step, layer:layer + 1]     # [1, q_heads, dim]
            serving.splitzip_qk_norm_rope(qr, kr, vr, m.norm[layer][0], m.norm[layer][1], position, m.table, first, q, new[0], new[1])
            paged.splitzip_pages_store(new[0], new[1], slots(layer, first + s.kept + step), pool)
            paged.splitzip_paged_attention(q, pool, table[layer:layer + 1], start, lens, out, workspace, 1)
            x = m.mix(layer, x, out)
    return outs, queries, pool, table


def run(s: Shape, device="cuda") -> dict:
    m = Layers(s, device)
    kv, weights = prefill(m)
    small, index = thin(s, kv, weights)
    payload, nbytes, there = send(s, small)
    if s.pages:
        outs, queries, decoded, table = decode_paged(m, there)
    else:
        (outs, queries, decoded), table = decode(m, there), None
    torch.cuda.synchronize()
    return {"kv": kv, "weights": weights, "small": small, "index": index, "there": there, "outs": outs,
            "queries": queries, "decoded": decoded, "table": table, "payload_bytes": nbytes, "layers": m}


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in vars(Shape()).items():
        ap.add_argument(f"--{name.replace('_', '-')}", type=type(value), default=value)
    s = Shape(**vars(ap.parse_args(argv)))
    r = run(s)
    bits = torch.int16 if s.fmt == "bf16" else torch.uint8
    same = torch.equal(r["small"].view(bits), r["there"].view(bits))
    whole, thinned = (t.numel() * t.element_size() for t in (r["kv"], r["small"]))
    print(f"{s.layers} layers, {s.tokens} tokens: cache {whole / 1e6:.1f} MB, thinned to {s.kept} tokens {thinned / 1e6:.1f} MB, "
          f"sent {r['payload_bytes'] / 1e6:.1f} MB ({whole / r['payload_bytes']:.2f}x less than the cache)")
    print(f"arrived bit for bit: {same}; {s.steps} tokens decoded, outputs finite: {bool(torch.isfinite(r['outs']).all())}")
    return 0 if same else 1


if __name__ == "__main__":
    raise SystemExit(main())
