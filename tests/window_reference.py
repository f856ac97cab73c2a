"""The window-attention operators from their definitions, in float64 on the CPU,
with elementwise error bounds of the GPU kernels.

Bounds.  As for the latent operators (latent_reference.py): a rounding to bf16 is
off by at most u = 2^-8 of the value, fp32 work by `SLACK` relative to the sum of
the magnitudes added (a score of d <= 128 products is off by at most 128 2^-24
scale sum|q k|, below 1e-4 for unit normal inputs if every error had the same
sign, and a weight is off by as much relatively).  The bf16 kernels round the
weights w before the product with the values, and dz before its products.

The norm: the sum of d <= 256 squares is off by at most 256 2^-24 = 1.5e-5
relatively, the root and the quotient by some 2^-24 more, an angle's cosine and
sine by 2^-22, a rotated element by those of both elements of its pair: within
SLACK (|a| + |b|) of the pair (a, b), with a factor of 5 to spare.
"""
from __future__ import annotations

import math

import torch

from latent_reference import SLACK, U, check, turned  # noqa: F401


def sees(n, m, window, sinks):
    """[n, m] which keys each query sees."""
    p = torch.arange(n)[:, None] + (m - n)
    j = torch.arange(m)[None]
    return (j <= p) & ((p - j < window) | (j < sinks))


def attention(q, k, v, lens_q, lens_k, window, sinks, scale=None, d_o=None, slack=SLACK):
    """dict name -> (value, bound) with o, lse and, given d_o, dq, dk, dv (rows of
    the sequences; rows behind them are zero)."""
    u = U[q.dtype]
    uw = u if q.dtype == torch.bfloat16 else 0.0     # rounding of the weights and dz
    scale = q.shape[2] ** -0.5 if scale is None else scale
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    T, H, d = q.shape
    Tk, Hk, _ = k.shape
    G = H // Hk
    z0 = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    out = {n: (z0(*s), z0(*s)) for n, s in (("o", (T, H, d)), ("lse", (T, H)), ("dq", (T, H, d)), ("dk", (Tk, Hk, d)),
                                            ("dv", (Tk, Hk, d)))}
    d_o = None if d_o is None else d_o.double().cpu()
    a = b = 0
    for n, m in zip(lens_q, lens_k):
        mask = sees(n, m, window, sinks)
        for h in range(H if n else 0):
            kh = h // G
            qs, ks, vs = q[a:a + n, h], k[b:b + m, kh], v[b:b + m, kh]
            z = (qs @ ks.t() * scale).masked_fill(~mask, -math.inf)
            lse = torch.logsumexp(z, dim=1) if m else torch.full((n,), -math.inf, dtype=torch.float64)
            w = torch.where(torch.isinf(lse)[:, None], torch.zeros_like(z), torch.exp(z - lse[:, None]))
            o = w @ vs
            eo = (uw + slack) * (w @ vs.abs()) + u * o.abs()
            out["o"][0][a:a + n, h], out["o"][1][a:a + n, h] = o, eo
            out["lse"][0][a:a + n, h] = lse
            out["lse"][1][a:a + n, h] = slack + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)
            if d_o is not None:
                g = d_o[a:a + n, h]
                delta = (g * o).sum(-1, keepdim=True)
                e_delta = (g.abs() * eo).sum(-1, keepdim=True)
                dz = w * (g @ vs.t() - delta)
                e_dz = w * (slack * (g.abs() @ vs.abs().t() + delta.abs()) + e_delta)
                e_all = (uw + slack) * dz.abs() + e_dz
                out["dv"][0][b:b + m, kh] += w.t() @ g
                out["dv"][1][b:b + m, kh] += (uw + slack) * (w.t() @ g.abs())
                out["dk"][0][b:b + m, kh] += dz.t() @ qs * scale
                out["dk"][1][b:b + m, kh] += e_all.t() @ qs.abs() * scale
                out["dq"][0][a:a + n, h] = dz @ ks * scale
                out["dq"][1][a:a + n, h] = e_all @ ks.abs() * scale
        a, b = a + n, b + m
    for name in ("dq", "dk", "dv"):
        out[name] = (out[name][0], out[name][1] + u * out[name][0].abs())
    if d_o is None:
        return {n: out[n] for n in ("o", "lse")}
    return out


def cached(cache, table, s, m):
    """The first m cached rows of sequence s (zeros where absent), and which are there."""
    P, page, Hk, d = cache.shape
    j = torch.arange(m)
    pg = table[s, j // page].long().cpu()
    there = (pg >= 0) & (pg < P)
    rows = torch.zeros(m, Hk, d, dtype=torch.float64)
    if there.any():
        rows[there] = cache[pg[there].to(cache.device), (j % page)[there].to(cache.device)].double().cpu()
    return rows, there


def decode(q, k_cache, v_cache, table, lens, new, window, sinks, scale=None):
    """(o, bound), (lse, bound) over the paged cache; pages outside the pool absent."""
    u = U[q.dtype]
    uw = u if q.dtype == torch.bfloat16 else 0.0
    scale = q.shape[2] ** -0.5 if scale is None else scale
    q = q.double().cpu()
    T, H, d = q.shape
    G = H // k_cache.shape[2]
    o, eo = torch.zeros(T, H, d, dtype=torch.float64), torch.zeros(T, H, d, dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    t = 0
    for s, (m, n) in enumerate(zip(lens, new)):
        m = max(0, min(m, table.shape[1] * k_cache.shape[1]))
        if m and n:
            (k, there), (v, _) = cached(k_cache, table, s, m), cached(v_cache, table, s, m)
            mask = sees(n, m, window, sinks) & there[None]
            # hidden rows may hold anything
            any_sees = mask.any(0)
            k, v = k.masked_fill(~any_sees[:, None, None], 0.0), v.masked_fill(~any_sees[:, None, None], 0.0)
            for h in range(H):
                z = (q[t:t + n, h] @ k[:, h // G].t() * scale).masked_fill(~mask, -math.inf)
                tot = torch.logsumexp(z, dim=1)
                w = torch.where(torch.isinf(tot)[:, None], torch.zeros_like(z), torch.exp(z - tot[:, None]))
                o[t:t + n, h] = w @ v[:, h // G]
                eo[t:t + n, h] = (uw + SLACK) * (w @ v[:, h // G].abs()) + u * o[t:t + n, h].abs()
                lse[t:t + n, h] = tot
        t += n
    return (o, eo), (lse, SLACK + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0))


def _part(x, fn, start, dr):
    y = x.clone()
    if dr:
        y[..., start:start + dr] = fn(x[..., start:start + dr].clone())
    return y


def _pair_size(x, interleaved):
    """|a| + |b| of every element's pair."""
    h = x.shape[-1] // 2
    y = torch.empty_like(x)
    if interleaved:
        s = x[..., 0::2].abs() + x[..., 1::2].abs()
        y[..., 0::2], y[..., 1::2] = s, s
    else:
        s = x[..., :h].abs() + x[..., h:].abs()
        y[..., :h], y[..., h:] = s, s
    return y


def norm(x, weight, positions, inv_freq, start, interleaved, eps=1e-6, amplitude=1.0, normalise=True):
    """(y, bound) of the norm and rotation of x [T, H, d]."""
    u = U[x.dtype]
    x = x.double().cpu()
    w = torch.ones(x.shape[2], dtype=torch.float64) if weight is None else weight.double().cpu()
    n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) if normalise else x
    y = n * w
    dr = 0 if inv_freq is None else 2 * inv_freq.numel()
    size = _part(y.abs(), lambda z: abs(amplitude) * _pair_size(z, interleaved), start, dr)
    y = _part(y, lambda z: turned(z, positions, inv_freq, interleaved, amplitude), start, dr)
    return y, u * y.abs() + SLACK * size


def norm_backward(x, dy, weight, positions, inv_freq, start, interleaved, eps=1e-6, amplitude=1.0):
    """(dx, bound), (dweight, bound)."""
    u = U[x.dtype]
    x, dy = x.double().cpu(), dy.double().cpu()
    w = torch.ones(x.shape[2], dtype=torch.float64) if weight is None else weight.double().cpu()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    n = x * r
    dr = 0 if inv_freq is None else 2 * inv_freq.numel()
    size = _part(dy.abs(), lambda z: abs(amplitude) * _pair_size(z, interleaved), start, dr)
    g = _part(dy, lambda z: turned(z, positions, inv_freq, interleaved, amplitude, inverse=True), start, dr)
    h = g * w
    dx = r * (h - n * (h * n).mean(-1, keepdim=True))
    e = SLACK * r * (size * w.abs() + n.abs() * (size * w.abs() * n.abs()).mean(-1, keepdim=True))
    return (dx, u * dx.abs() + e), ((g * n).sum((0, 1)), SLACK * (size * n.abs()).sum((0, 1)))
