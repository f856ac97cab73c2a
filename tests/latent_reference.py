"""The latent-attention operators from their definitions, in float64 on the
CPU, with elementwise error bounds of the GPU kernels.

Bounds.  A rounding to bf16 is off by at most u = 2^-8 of the value; fp32
outputs are rounded by 2^-24, which the slack covers.  The bf16 kernels round
the softmax weights w before the product with the values, and dz (the
gradient of the scores) before its products; everything else they hold in
fp32.  The fp32 work is off by `SLACK` relative to the sum of the magnitudes
added: a score of dqk <= 576 products is off by at most dqk 2^-24 scale
sum|q k|, about 1e-4 for unit normal inputs at dqk = 192 if every error had
the same sign, and a weight is off by as much relatively.  So, elementwise:
  o      u sum w|v| (weights) + u |o| (output)            + SLACK sum w|v|
  delta  sum |g| (error of o)
  dz     SLACK w (|g.v| + |delta|) + w (error of delta)   =: e_dz
  dv     u sum w|g| + u |dv|                              + SLACK sum w|g|
  dq     scale sum (u |dz| + e_dz) |k| + u |dq|           + SLACK scale sum |dz||k|
and dk like dq.
"""
from __future__ import annotations

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SLACK = 1e-4


def attention(q, k, v, k_pe, lens_q, lens_k, causal, scale, d_o=None, slack=SLACK):
    """Per sequence and head.  Returns a dict name -> (value, bound) with o,
    lse and, given d_o, dq, dk, dv, dk_pe (rows of the sequences; rows behind
    them are zero)."""
    dt = q.dtype
    u = U[dt]
    uw = u if dt == torch.bfloat16 else 0.0     # rounding of the weights and dz
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    dr = 0 if k_pe is None else k_pe.shape[1]
    if dr:
        k_pe = k_pe.double().cpu()
        k = torch.cat([k, k_pe[:, None].expand(-1, k.shape[1], -1)], dim=2)
    T, H, dqk = q.shape
    Tk, _, dv = v.shape
    dn = dqk - dr
    z0 = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    out = {n: (z0(*s), z0(*s)) for n, s in (("o", (T, H, dv)), ("lse", (T, H)), ("dq", (T, H, dqk)),
                                            ("dk", (Tk, H, dqk)), ("dv", (Tk, H, dv)))}
    d_o = None if d_o is None else d_o.double().cpu()
    a = b = 0
    for n, m in zip(lens_q, lens_k):
        if n:
            qs, ks, vs = (x.transpose(0, 1) for x in (q[a:a + n], k[b:b + m], v[b:b + m]))
            z = (qs @ ks.transpose(1, 2)) * scale
            if causal:
                i, j = torch.arange(n)[:, None], torch.arange(m)[None]
                z = z.masked_fill(j > i + (m - n), -math.inf)
            lse = torch.logsumexp(z, dim=2) if m else torch.full((H, n), -math.inf, dtype=torch.float64)
            w = torch.where(torch.isinf(lse)[..., None], torch.zeros_like(z), torch.exp(z - lse[..., None]))
            o = w @ vs
            wv = w @ vs.abs()
            eo = (uw + slack) * wv + u * o.abs()
            out["o"][0][a:a + n], out["o"][1][a:a + n] = o.transpose(0, 1), eo.transpose(0, 1)
            out["lse"][0][a:a + n] = lse.transpose(0, 1)
            out["lse"][1][a:a + n] = (slack + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)).transpose(0, 1)
            if d_o is not None:
                g = d_o[a:a + n].transpose(0, 1)
                delta = (g * o).sum(-1, keepdim=True)
                e_delta = (g.abs() * eo).sum(-1, keepdim=True)
                gv = g @ vs.transpose(1, 2)
                dz = w * (gv - delta)
                # |g| . |v| bounds the fp32 sum of g . v and of delta
                mag = g.abs() @ vs.abs().transpose(1, 2)
                e_dz = w * (slack * (mag + delta.abs()) + e_delta)
                for name, x, e in (("dv", w.transpose(1, 2) @ g, (uw + slack) * (w.transpose(1, 2) @ g.abs())),
                                   ("dk", dz.transpose(1, 2) @ qs * scale,
                                    ((uw + slack) * dz.abs() + e_dz).transpose(1, 2) @ qs.abs() * scale)):
                    out[name][0][b:b + m], out[name][1][b:b + m] = x.transpose(0, 1), e.transpose(0, 1)
                out["dq"][0][a:a + n] = (dz @ ks * scale).transpose(0, 1)
                out["dq"][1][a:a + n] = (((uw + slack) * dz.abs() + e_dz) @ ks.abs() * scale).transpose(0, 1)
        a, b = a + n, b + m
    for name in ("dq", "dk", "dv"):
        out[name] = (out[name][0], out[name][1] + u * out[name][0].abs())
    x, e = out["dk"]
    out["dk"] = (x[..., :dn], e[..., :dn])
    if dr:
        pe = x[..., dn:].sum(1)
        out["dk_pe"] = (pe, (e[..., dn:] - u * x[..., dn:].abs()).sum(1) + u * pe.abs())
    return out


def decode(q, cache, table, lens, new, dl, scale):
    """Absorbed attention over the paged cache: (o, bound), (lse, bound); rows
    of packed new tokens, pages outside the pool absent."""
    dt = q.dtype
    u = U[dt]
    uw = u if dt == torch.bfloat16 else 0.0
    q, table = q.double().cpu(), table.cpu()
    P, page, _ = cache.shape
    T, H, _ = q.shape
    o, eo = torch.zeros(T, H, dl, dtype=torch.float64), torch.zeros(T, H, dl, dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    t = 0
    for s, (m, n) in enumerate(zip(lens, new)):
        m = max(0, min(m, table.shape[1] * page))
        j = torch.arange(m)
        pg = table[s, j // page].long()
        there = (pg >= 0) & (pg < P)
        rows = torch.zeros(m, cache.shape[2], dtype=torch.float64)
        if there.any():
            at = (pg * page + j % page)[there].to(cache.device)
            rows[there] = cache.reshape(-1, cache.shape[2])[at].double().cpu()
        for i in range(n):
            z = (q[t + i] @ rows.t()) * scale
            z = z.masked_fill(~there[None] | (j > m - n + i)[None], -math.inf)
            tot = torch.logsumexp(z, dim=1) if m else torch.full((H,), -math.inf, dtype=torch.float64)
            w = torch.where(torch.isinf(tot)[:, None], torch.zeros_like(z), torch.exp(z - tot[:, None]))
            o[t + i] = w @ rows[:, :dl]
            eo[t + i] = (uw + SLACK) * (w @ rows[:, :dl].abs()) + u * o[t + i].abs()
            lse[t + i] = tot
        t += n
    return (o, eo), (lse, SLACK + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0))


def turned(x, positions, inv_freq, interleaved, amplitude=1.0, inverse=False):
    """Pairs of the last axis of x [T, ..., dr] rotated by position * frequency."""
    x = x.double().cpu()
    h = x.shape[-1] // 2
    ang = positions.double().cpu()[:, None] * inv_freq.double().cpu()[None]
    ang = ang.reshape(ang.shape[0], *([1] * (x.dim() - 2)), h)
    c, s = torch.cos(ang) * amplitude, torch.sin(ang) * amplitude * (-1.0 if inverse else 1.0)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    y = torch.empty_like(x)
    p, r = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0::2], y[..., 1::2] = p, r
    else:
        y[..., :h], y[..., h:] = p, r
    return y


def check(label, got, want, bound):
    """Elementwise |got - want| <= bound; infinities equal."""
    got = got.detach().double().cpu()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and not torch.isnan(got).any(), f"{label}: non-finite values differ"
    assert torch.equal(got[inf], want[inf]), f"{label}: infinities differ"
    err = (got - want).abs().masked_fill(inf, 0.0)
    over = err - bound.masked_fill(inf, 0.0)
    den = float(want[~inf].norm())
    rel = float(err.norm()) / den if den > 0 else float(err.norm())
    worst = float(over.max()) if over.numel() else 0.0
    print(f"[latent] {label}: rel-L2 {rel:.2e}, largest excess over the bound {worst:.2e}", flush=True)
    assert worst <= 1e-30, f"{label}: off by more than the bound, excess {worst:.3e}"
    return rel
