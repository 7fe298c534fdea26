"""The paged cache's operators in 64 bits, written from their definitions
(include/splitzip_pages.h).  Small sizes only."""
import math

import torch

from tests import serving_ref

#: of a format: its codes' magnitudes, half way from the largest to where a larger one
#: would be, and the powers that the store uses
GRID = {"int8": ([float(i) for i in range(128)], 127.5, -24, 9),
        "e2m1": ([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], 7.0, -23, 13)}
QUANTISED = tuple(GRID)


def two_to(k):
    """2^k in 64 bits, k an integer tensor."""
    return (k.long() + 1023 << 52).view(torch.float64)


def quantise(x, fmt):
    """(signed code numbers' magnitudes index, sign, exponent bytes [..., 4]) of BF16 rows [..., dim]."""
    if x.numel() > 1 << 22 and len(x) > 1:      # half at a time: the table of distances is large
        return tuple(map(torch.cat, zip(*(quantise(half, fmt) for half in x.tensor_split(2)))))
    grid, beyond, low, high = GRID[fmt]
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    v = x.double().unflatten(-1, (4, -1))
    most = v.abs().amax(-1)
    odd = ~torch.isfinite(v).all(-1)
    k = torch.full(most.shape, low, device=x.device)
    for p in range(low, high):
        k = torch.where(most >= beyond * 2.0 ** p, p + 1, k)
    z = torch.where(odd[..., None], 0.0, v) / two_to(k)[..., None]
    far = (z.abs().clamp_max(grid[-1])[..., None] - grid).abs()
    best = far.amin(-1, keepdim=True)
    near = far == best                       # one, or two at a tie: the even one of them
    index = torch.arange(len(grid), device=x.device)
    code = torch.where(near, index + 1000 * (index % 2), 10 ** 6).amin(-1)
    code = torch.where(code >= 1000, code - 1000, code)
    exps = torch.where(odd, 255, torch.where(most == 0, 0, k + 127)).to(torch.uint8)
    return code.flatten(-2), torch.signbit(z).flatten(-2), exps


def codes(x, fmt):
    """What the store writes for BF16 rows: (stored row, exponent bytes or None)."""
    if fmt == "bf16":
        return x, None
    if fmt == "e5m2":
        return x.float().to(torch.float8_e5m2), None
    code, neg, exps = quantise(x, fmt)
    if fmt == "int8":
        return torch.where(neg, -code, code).to(torch.int8), exps
    nibble = (code + 8 * neg).to(torch.uint8)
    return nibble[..., 0::2] + 16 * nibble[..., 1::2], exps


def values(rows, exps, fmt):
    """Stored rows in 64 bits."""
    if fmt in ("bf16", "e5m2"):
        return rows.double()
    if fmt == "int8":
        z = rows.double()
    else:
        n = torch.stack([rows % 16, rows // 16], -1).flatten(-2).long()
        z = torch.tensor(GRID["e2m1"][0], dtype=torch.float64, device=rows.device)[n % 8]
        z = torch.where(n >= 8, -z, z)
    scale = torch.where(exps == 255, math.nan, torch.where(exps == 0, 0.0, two_to(exps.long() - 127)))
    return (z.unflatten(-1, (4, -1)) * scale[..., None]).flatten(-2)


def sequence(pages, table_row, n, which="k"):
    """[n, heads, dim] in 64 bits: one sequence of a pool, NaN where its page is outside."""
    fmt = {torch.bfloat16: "bf16", torch.float8_e5m2: "e5m2", torch.int8: "int8", torch.uint8: "e2m1"}[pages.k.dtype]
    t = torch.arange(n, device=table_row.device)
    page, at = table_row.long()[t // pages.page_tokens], t % pages.page_tokens
    ok = (page >= 0) & (page < pages.pages)
    page = torch.where(ok, page, 0)
    exps = getattr(pages, which + "_exp")
    rows = getattr(pages, which)
    rows = rows.view(torch.uint8)[page, at].view(rows.dtype) if fmt == "e5m2" else rows[page, at]
    v = values(rows, None if exps is None else exps[page, at], fmt)
    return torch.where(ok[:, None, None], v, math.nan)


def attention(q, pages, table, q_start, lens, kv_tokens, window, sinks, scale):
    """[(rows of q, out, lse [heads, rows], tolerance of both)], one for each sequence with new tokens.

    Bounds: those of serving_ref.attention (whose 2^-8 of each weight covers the 2^-11 of FP16), and for caches
    other than BF16 what FP16 weights lose at the lower end.  FP16 numbers below 2^-14 are 2^-24 apart, so a
    weight is off by at most 2^-25; a row's largest weight then is at least 2^8 (the kernels take 2^8 to 2^9, or
    2^15, for it), so that is 2^-33 of the largest, which is at most 1 of the sum: 2^-33 of the sum of the seen
    |v| in all.  It counts where values are 0 at all large weights, as quantised ones often are."""
    found = []
    fine = 0.0 if pages.k.dtype == torch.bfloat16 else 2.0 ** -33
    starts = q_start.tolist()
    for b, n in enumerate(lens.clamp(0, kv_tokens).tolist()):
        i, j = starts[b], starts[b + 1]
        if i == j:
            continue
        k, v = (sequence(pages, table[b], n, x)[None] for x in "kv")
        if n == 0:      # nothing to see: one slot that is masked
            k = v = torch.zeros((1, 1, *pages.k.shape[2:3], q.shape[2]), dtype=torch.float64, device=q.device)
        o, l, tol, ltol = serving_ref.attention(q[None, i:j], k, v, torch.tensor([n], device=q.device), window, sinks, scale)
        size = torch.where(v.isfinite(), v.abs(), 0.0).sum(1)[0]     # [kv_heads, dim]
        tol = tol[0] + fine * size.repeat_interleave(q.shape[1] // size.shape[0], 0)
        found.append((slice(i, j), o[0], l[0], tol, ltol[0]))
    return found
