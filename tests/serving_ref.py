"""The operators around the KV cache in 64 bits, written from their definitions
(include/splitzip_serving.h), with the error bounds the tests hold the library
to.  Small sizes only: every score is materialised."""
import math

import torch


def visible(lens, q_tokens, kv_tokens, window, sinks):
    """bool [batch, q_tokens, kv_tokens]."""
    dev = lens.device
    p = lens.long()[:, None, None] - q_tokens + torch.arange(q_tokens, device=dev)[None, :, None]
    t = torch.arange(kv_tokens, device=dev)[None, None, :]
    see = t <= p
    if window:
        see = see & ((t > p - window) | (t < sinks))
    return see


def scores(q, k, scale):
    """(scores, sums of magnitudes) [batch, kv_heads, group, q_tokens, kv_tokens]."""
    b, tq, hq, d = q.shape
    hk = k.shape[2]
    qd = q.double().view(b, tq, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    kd = k.double().permute(0, 2, 3, 1)[:, :, None]
    return qd @ kd * scale, qd.abs() @ kd.abs() * abs(scale)


def attention(q, k, v, lens, window, sinks, scale):
    """out [b, tq, hq, d], lse [b, hq, tq], and bounds of the errors of both.

    Bounds: a score is a 32-bit sum of d products, off by at most d 2^-23 of the
    sum of magnitudes (gamma); exp turns that into a relative error of each
    weight, twice (numerator and sum).  The weights enter the second product in
    16 bits, 2^-8 of each (BF16 has 8 significant bits: half a step is at most
    2^-8 of the value); the result is rounded once to BF16, 2^-8 of it.
    2^-13 covers the exponential's and the sums' own 32-bit rounding and the
    scaling of scores of up to 2^8."""
    b, tq, hq, d = q.shape
    hk = k.shape[2]
    see = visible(lens, tq, k.shape[1], window, sinks)[:, None, None]
    s, mag = scores(q, k, scale)
    gamma = (torch.where(see, mag, 0.0).amax(-1, keepdim=True) * d * 2.0 ** -23)
    s = torch.where(see, s, -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.where(see, torch.exp(s - torch.where(lse > -math.inf, lse, 0.0)), 0.0)
    vd = v.double().permute(0, 2, 1, 3)[:, :, None]
    ok = vd.isfinite()
    o = p @ torch.where(ok, vd, 0.0)
    mass = p @ torch.where(ok, vd.abs(), 0.0)
    if not bool(ok.all()):   # what a visible infinity or NaN makes of the sum
        odd = torch.where(ok, 0.0, vd)
        for t in (~ok).any(-1).any(2).any(1).any(0).nonzero().flatten().tolist():
            o = o + torch.where(see[..., t, None], odd[..., t, :].unsqueeze(-2), 0.0)
    tol = o.abs() * 2.0 ** -8 + mass * (2.0 ** -8 + 2.0 ** -13 + 2 * gamma) + 1e-30
    shape = lambda x: x.permute(0, 3, 1, 2, 4).reshape(b, tq, hq, d)  # noqa: E731
    lse_tol = gamma + lse.abs().nan_to_num(posinf=0.0) * 2.0 ** -21 + 2.0 ** -20
    return shape(o), lse.view(b, hq, tq), shape(tol), lse_tol.view(b, hq, tq)


def weights(q, k, lse, lens, window, sinks, scale, before=None):
    """(weights [b, hk, tk], bound).  Bound: each term is off by its score's error
    and its exponent's 32-bit rounding, 2^-23 of up to 2^5 times 2 roundings; a
    sum of N positive terms in 32 bits by at most N 2^-24 of itself."""
    b, tq, hq, d = q.shape
    hk = k.shape[2]
    see = visible(lens, tq, k.shape[1], window, sinks)[:, None, None]
    s, mag = scores(q, k, scale)
    gamma = torch.where(see, mag, 0.0).max() * d * 2.0 ** -23
    l = lse.double().view(b, hk, hq // hk, tq, 1)
    w = torch.where(see, torch.exp(s - torch.where(l > -math.inf, l, 0.0)), 0.0).sum((2, 3))
    tol = w * (gamma + 2.0 ** -17 + tq * (hq // hk) * 2.0 ** -24) + 1e-30
    if before is not None:
        w = w + before.double()
    return w, tol + w.abs() * 2.0 ** -23


def norm_rope(x, weight, positions, table, eps, interleaved):
    """(rows, bound without the last rounding) of [n, heads, d]: every product and
    sum is a 32-bit one, a few 2^-23 of the pair's magnitudes."""
    y = x.double()
    y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    r = 0 if table is None else table.shape[1]
    size = y.abs()
    if r:
        t = table.double()[positions.long()][:, None]
        c, s = t[..., : r // 2], t[..., r // 2:]
        if interleaved:
            c, s = c.repeat_interleave(2, -1), s.repeat_interleave(2, -1)
            partner = y[..., :r].unflatten(-1, (r // 2, 2)).flip(-1).flatten(-2)
            sign = torch.tensor([-1.0, 1.0], device=x.device).double().repeat(r // 2)
        else:
            c, s = torch.cat([c, c], -1), torch.cat([s, s], -1)
            partner = torch.cat([y[..., r // 2: r], y[..., : r // 2]], -1)
            sign = torch.cat([-torch.ones(r // 2), torch.ones(r // 2)]).double().to(x.device)
        size = torch.cat([y[..., :r].abs() + partner.abs(), y[..., r:].abs()], -1)
        y = torch.cat([y[..., :r] * c + sign * partner * s, y[..., r:]], -1)
    return y, size * 2.0 ** -19


def evict_slots(w, n, budget, first, last):
    """Kept slots of one head (python list of weights): the definition, sorted."""
    if n <= budget:
        return list(range(n))
    always = set(range(first)) | set(range(n - last, n))
    rest = [i for i in range(n) if i not in always]
    rest.sort(key=lambda i: (1, 0.0, i) if math.isnan(w[i]) else (0, -w[i], i))
    return sorted(always | set(rest[: budget - first - last]))
