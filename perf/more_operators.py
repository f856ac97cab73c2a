"""Measurement cases of the sliding-window attention operators: what they
compute in plain torch operations, and the calls a program makes of the library
instead.

A local attention layer beside KDA layers lets a token see the last ``window``
tokens, itself included, and the first few of the sequence (``sinks``).  H query
heads share Hk key and value heads.  Four operators serve it:

  attn, train  packed sequences: the forward pass, and a training step with the
               gradients of q, k and v;
  decode       one or more new tokens per sequence over a paged cache of keys
               and values;
  append       the new tokens' keys (normalised per head, rotated) and values
               written to their places in that cache;
  norm         queries and keys normalised per head and rotated in one pass,
               forward, and as a training step with the gradients of both and
               of the norms' weights.

``own`` selects the library's calls; otherwise ``run`` computes the plain form
in 32 bits, rounded once at the end.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# -- cases ---------------------------------------------------------------------

def _text(lens):
    return ",".join(str(int(x)) for x in lens)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _uniform(seed, n, lo, hi):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(n)]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def listed():
    return [
        # a handful of short ragged prompts in fp32: a unit test's or a small model's prefill, latency bound
        dict(name="attn-f32-ragged", kind="attn", dtype="f32", H=8, Hk=2, d=64, lens="1,130,17,64,77,5", prefix=0,
             window=32, sinks=4),
        # one long prompt of a full-size layer: 32,768 tokens, 32 query and 8 key heads of 128 channels
        dict(name="attn-bf16-32768", kind="attn", dtype="bf16", H=32, Hk=8, d=128, lens="32768", prefix=0,
             window=4096, sinks=4),
        # a small fp32 training step over ragged documents (gradient checks, small models)
        dict(name="train-f32-ragged", kind="train", dtype="f32", H=4, Hk=2, d=128, lens="300,1,65,129", prefix=0,
             window=100, sinks=2),
        # a training step of a full-size layer over 16 packed documents of 256 to 4,096 tokens
        dict(name="train-bf16-packed16", kind="train", dtype="bf16", H=32, Hk=8, d=128,
             lens=_text(_uniform(3, 16, 256, 4096)), prefix=0, window=1024, sinks=4),
        # one sequence alone, 65,536 tokens in the cache, one new token: the latency of long-context decoding
        dict(name="decode-one-65536", kind="decode", dtype="bf16", H=32, Hk=8, d=128, page=64, lens="65536", new="1",
             window=4096, sinks=4),
        # the serving batch: 256 sequences of 256 to 8,192 tokens, one new token each
        dict(name="decode-256", kind="decode", dtype="bf16", H=32, Hk=8, d=128, page=64,
             lens=_text(_uniform(7, 256, 256, 8192)), new=_text([1] * 256), window=1024, sinks=4),
        # chunks of 128 new tokens of 16 prompts over their cached prefixes (chunked prefill, resumed prefixes)
        dict(name="decode-chunk-16x128", kind="decode", dtype="bf16", H=32, Hk=8, d=128, page=64,
             lens=_text(_uniform(6, 16, 1024, 4096)), new=_text([128] * 16), window=1024, sinks=4),
        # a small fp32 cache: short sequences, small pages, one to three new tokens (speculative checks)
        dict(name="decode-f32-small", kind="decode", dtype="f32", H=8, Hk=2, d=64, page=16, lens="200,1,77,333",
             new="1,1,3,2", window=64, sinks=4),
        # the cache write of one serving step: 256 sequences, one token each
        dict(name="append-step-256", kind="append", dtype="bf16", Hk=8, d=128, dr=128, page=64,
             lens=_text(_uniform(7, 256, 256, 8192)), new=_text([1] * 256), interleaved=False, norm=True, outs=False),
        # the cache write of 16 whole prompts, which also keeps the keys for the prompts' own attention
        dict(name="append-prompts-16", kind="append", dtype="bf16", Hk=8, d=128, dr=64, page=64,
             lens=_text(_uniform(3, 16, 256, 4096)), new=_text(_uniform(3, 16, 256, 4096)), interleaved=True,
             norm=True, outs=True),
        # queries and keys of one serving step: 256 tokens at far positions
        dict(name="norm-step-256", kind="norm", dtype="bf16", T=256, H=32, Hk=8, d=128, start=0, dr=128,
             interleaved=False, far=1000000, train=False),
        # queries and keys of a training step over 36,755 tokens, half of the channels rotated, with all gradients
        dict(name="norm-train-36755", kind="norm", dtype="bf16", T=36755, H=32, Hk=8, d=128, start=0, dr=64,
             interleaved=False, far=4096, train=True),
    ]


def _draw_heads(rng):
    Hk = rng.choice([1, 2, 3, 4, 8])
    return Hk * rng.choice([1, 2, 4, 5, 8]), Hk


def _draw_attention(rng):
    train = rng.random() < 0.5
    f32 = rng.random() < 0.3
    H, Hk = _draw_heads(rng)
    total = _log_int(rng, 16, 2048 if f32 else 16384)
    n = min(total, _log_int(rng, 1, 24))
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    # now and then keys longer than the queries: new tokens after a kept prefix
    prefix = _log_int(rng, 1, 1024) if rng.random() < 0.25 else 0
    return dict(kind="train" if train else "attn", dtype="f32" if f32 else "bf16", H=H, Hk=Hk,
                d=rng.choice([64, 128]), lens=_text(lens), prefix=prefix, window=_log_int(rng, 1, 4096),
                sinks=rng.choice([0, 0, 1, 4, 17, 64]))


def _draw_decode(rng):
    f32 = rng.random() < 0.25
    H, Hk = _draw_heads(rng)
    n = _log_int(rng, 1, 32 if f32 else 256)
    hi = _log_int(rng, 1, max(2, min(65536, (40000 if f32 else 800000) // n)))
    lens = [rng.randint(max(1, hi // 8), hi) for _ in range(n)]
    window = _log_int(rng, 1, 1024 if n > 64 else 4096)
    if rng.random() < 0.5:
        new = [1] * n
    else:
        most = _log_int(rng, 1, max(1, min(256, 4096 // n)))
        new = [rng.randint(1, min(most, x)) for x in lens]
    return dict(kind="decode", dtype="f32" if f32 else "bf16", H=H, Hk=Hk, d=rng.choice([64, 128]),
                page=rng.choice([1, 16, 48, 64, 128]), lens=_text(lens), new=_text(new), window=window,
                sinks=rng.choice([0, 0, 1, 4, 17, 64]))


def _draw_append(rng):
    n = _log_int(rng, 1, 256)
    hi = _log_int(rng, 1, max(1, 30000 // n))
    new = [rng.randint(1, hi) for _ in range(n)] if rng.random() < 0.5 else [1] * n
    lens = [x + _log_int(rng, 1, 2048) - 1 for x in new]
    d = rng.choice([64, 128])
    return dict(kind="append", dtype=rng.choice(["bf16", "bf16", "f32"]), Hk=_draw_heads(rng)[1], d=d,
                dr=rng.choice([0, 32, d]), page=rng.choice([1, 16, 48, 64, 128]), lens=_text(lens), new=_text(new),
                interleaved=rng.random() < 0.5, norm=rng.random() < 0.7, outs=rng.random() < 0.5)


def _draw_norm(rng):
    H, Hk = _draw_heads(rng)
    d = rng.choice([64, 80, 128, 256])
    dr = rng.choice([32, 64, d])
    return dict(kind="norm", dtype=rng.choice(["bf16", "bf16", "f32"]), T=_log_int(rng, 1, 16384), H=H, Hk=Hk, d=d,
                start=rng.choice([0, d - dr]), dr=dr, interleaved=rng.random() < 0.5, far=_log_int(rng, 1, 4000000),
                train=rng.random() < 0.6)


def draw(rng):
    return rng.choice([_draw_attention, _draw_attention, _draw_decode, _draw_decode, _draw_append, _draw_norm])(rng)


# -- inputs --------------------------------------------------------------------

def _offsets(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return at


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    def weight(d):
        return 1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")

    def freq(dr):
        return (500000.0 ** (-torch.arange(0, dr, 2, dtype=torch.float64) / dr)).float().cuda()

    s = dict(case=case)
    d = case["d"]
    if case["kind"] == "norm":
        T, H, Hk = case["T"], case["H"], case["Hk"]
        s["qkv"] = normal(T, H + 2 * Hk, d)              # what the projection leaves: queries, keys, values
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"] = freq(case["dr"])
        s["q_weight"], s["k_weight"] = weight(d), weight(d)
        if case["train"]:
            s["dq"], s["dk"] = normal(T, H, d), normal(T, Hk, d)
        return s
    lens = _ints(case["lens"])
    n = len(lens)
    if case["kind"] in ("attn", "train"):
        H, Hk = case["H"], case["Hk"]
        lens_k = [x + case["prefix"] for x in lens]
        T, Tk = sum(lens), sum(lens_k)
        # queries of unequal sharpness from head to head, as trained heads have
        sharp = 0.5 + 1.5 * torch.rand(H, 1, generator=g, device="cuda")
        s["q"] = (torch.randn(T, H, d, generator=g, device="cuda") * sharp).to(dt)
        s["kv"] = normal(Tk, 2 * Hk, d)                  # keys, then values of one projection
        s["lens"], s["lens_k"] = lens, lens_k
        s["cu_q"] = torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda")
        s["cu_k"] = torch.tensor(_offsets(lens_k), dtype=torch.int32, device="cuda") if case["prefix"] else s["cu_q"]
        if case["kind"] == "train":
            s["d_o"] = normal(T, H, d)
        return s
    new = _ints(case["new"])
    Hk, page = case["Hk"], case["page"]
    T = sum(new)
    used = [-(-x // page) for x in lens]
    pages = sum(used) + sum(used) // 8 + 1                # a pool with some pages free
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, max(used)), -1, dtype=torch.int32).cuda()
    place = torch.cat([torch.full((u,), i, dtype=torch.int64) for i, u in enumerate(used)])
    column = torch.cat([torch.arange(u) for u in used])
    table[place.cuda(), column.cuda()] = order[:sum(used)]
    s["block_table"] = table
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu_seqlens"] = torch.tensor(_offsets(new), dtype=torch.int32, device="cuda")
    s["lens"], s["new"] = lens, new
    for name in ("k_cache", "v_cache"):
        s[name] = torch.empty(pages, page, Hk, d, dtype=dt, device="cuda")
        step = max(1, (1 << 25) // (page * Hk * d))       # filled in pieces: the fp32 draw of a large pool is as large again
        for a in range(0, pages, step):
            s[name][a:a + step] = normal(min(pages, a + step) - a, page, Hk, d)
    if case["kind"] == "decode":
        s["q"] = normal(T, case["H"], d)
        return s
    s["kv"] = normal(T, 2 * Hk, d)                        # keys, then values of one projection
    s["norm_weight"] = weight(d) if case["norm"] else None
    s["inv_freq"] = freq(case["dr"]) if case["dr"] else None
    return s


# -- one pass --------------------------------------------------------------------

def run(state):
    return {"attn": _attention, "train": _train, "decode": _decode, "append": _append,
            "norm": _norm}[state["case"]["kind"]](state)


BLOCK = 1024   # query rows whose scores the plain form holds at a time


def _pieces(s):
    """Blocks of queries with the keys they see, [a, a + n) of the packed queries and their keys' rows: the first
    sinks and a run behind them, with which of the pairs are visible."""
    c = s["case"]
    W, S = c["window"], c["sinks"]
    a0 = b0 = 0
    for n, m in zip(s["lens"], s["lens_k"]):
        for i in range(0, n, BLOCK):
            cnt = min(BLOCK, n - i)
            p = torch.arange(i, i + cnt, device="cuda").unsqueeze(1) + (m - n)
            lo, hi = max(0, i + m - n - W + 1), i + cnt + m - n
            lo = max(lo, min(S, hi))
            j = torch.cat([torch.arange(0, min(S, hi), device="cuda"), torch.arange(lo, hi, device="cuda")])
            yield a0 + i, cnt, b0 + j, (j <= p) & ((p - j < W) | (j < S))
        a0, b0 = a0 + n, b0 + m


def _grouped(x, Hk):
    """[n, H, d] as fp32 [Hk, H / Hk * n, d]: the rows that share a key head."""
    n, H, d = x.shape
    return x.float().reshape(n, Hk, H // Hk, d).permute(1, 2, 0, 3).reshape(Hk, H // Hk * n, d)


def _ungrouped(x, n):
    Hk, _, d = x.shape
    return x.reshape(Hk, -1, n, d).permute(2, 0, 1, 3).reshape(n, -1, d)


def _probabilities(q, k, sees, scale):
    """softmax over the visible keys, and the log of its sum; q [Hk, G n, d], k [Hk, m, d], sees [n, m]."""
    p = (q @ k.transpose(1, 2)).mul_(scale)
    n, m = sees.shape
    p = p.reshape(p.shape[0], -1, n, m).masked_fill_(~sees, -math.inf)
    top = p.amax(dim=3, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(dim=3, keepdim=True)
    p.div_(total)
    return p.reshape(p.shape[0], -1, m), (top + total.log()).squeeze(3)


def _attention(s):
    c = s["case"]
    k, v = s["kv"][:, :c["Hk"]], s["kv"][:, c["Hk"]:]
    if own:
        import gated_delta_rule_prefill_amd as kda
        o, lse = kda.window_attention(s["q"], k, v, window=c["window"], sinks=c["sinks"], cu_seqlens=s["cu_q"],
                                      cu_seqlens_k=s["cu_k"])
        return {"o": o, "lse": lse}
    T, H, d = s["q"].shape
    o = torch.empty_like(s["q"])
    lse = torch.empty(T, H, device="cuda")
    for a, n, rows, sees in _pieces(s):
        ks, vs = k[rows].float().transpose(0, 1), v[rows].float().transpose(0, 1)
        p, l = _probabilities(_grouped(s["q"][a:a + n], c["Hk"]), ks, sees, d ** -0.5)
        o[a:a + n] = _ungrouped(p @ vs, n).to(o.dtype)
        lse[a:a + n] = l.permute(2, 0, 1).reshape(n, H)
    return {"o": o, "lse": lse}


def _train(s):
    c = s["case"]
    Hk = c["Hk"]
    k, v = s["kv"][:, :Hk], s["kv"][:, Hk:]
    if own:
        import gated_delta_rule_prefill_amd as kda
        args = dict(window=c["window"], sinks=c["sinks"], cu_seqlens=s["cu_q"], cu_seqlens_k=s["cu_k"])
        o, lse = kda.window_attention(s["q"], k, v, **args)
        g = kda.window_attention_backward(s["q"], k, v, o, lse, s["d_o"], **args)
        return {"o": o, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}
    scale, dt = c["d"] ** -0.5, s["q"].dtype
    o, dq = torch.empty_like(s["q"]), torch.empty_like(s["q"])
    dk, dv = (torch.zeros(k.shape, device="cuda") for _ in range(2))
    for a, n, rows, sees in _pieces(s):
        qs, gs = _grouped(s["q"][a:a + n], Hk), _grouped(s["d_o"][a:a + n], Hk)
        ks, vs = k[rows].float().transpose(0, 1), v[rows].float().transpose(0, 1)
        p, _ = _probabilities(qs, ks, sees, scale)
        os = p @ vs
        o[a:a + n] = _ungrouped(os, n).to(dt)
        dv.index_add_(0, rows, (p.transpose(1, 2) @ gs).transpose(0, 1))
        ds = (gs @ vs.transpose(1, 2)).sub_((gs * os).sum(dim=2, keepdim=True)).mul_(p).mul_(scale)
        dq[a:a + n] = _ungrouped(ds @ ks, n).to(dt)
        dk.index_add_(0, rows, (ds.transpose(1, 2) @ qs).transpose(0, 1))
    return {"o": o, "dq": dq, "dk": dk.to(dt), "dv": dv.to(dt)}


def _decode(s):
    c = s["case"]
    if own:
        import gated_delta_rule_prefill_amd as kda
        o, lse = kda.window_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                                   window=c["window"], sinks=c["sinks"], cu_seqlens=s["cu_seqlens"])
        return {"o": o, "lse": lse}
    T, H, d = s["q"].shape
    Hk, W, S, page = c["Hk"], c["window"], c["sinks"], c["page"]
    n, many = len(s["lens"]), max(s["new"])
    # the keys that a sequence's new tokens may see, padded to the longest: its sinks and its last W + many - 1 tokens
    span = min(max(s["lens"]), W + many - 1)
    lens = s["seq_lens"].long().unsqueeze(1)
    lo = (lens - span).clamp(min=S)                       # where the run behind the sinks starts
    j = torch.cat([torch.arange(S, device="cuda").expand(n, S), lo + torch.arange(span, device="cuda")], dim=1)
    there = j < lens
    j = torch.where(there, j, torch.zeros_like(j))
    rows = s["block_table"].long().gather(1, j // page) * page + j % page
    k = s["k_cache"].reshape(-1, Hk, d)[rows].float().transpose(1, 2)       # [n, Hk, keys, d]
    v = s["v_cache"].reshape(-1, Hk, d)[rows].float().transpose(1, 2)
    new = (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).long().unsqueeze(1)
    i = torch.arange(many, device="cuda")
    at = torch.where(i < new, s["cu_seqlens"][:-1].long().unsqueeze(1) + i, torch.zeros_like(new))
    q = s["q"].float()[at].reshape(n, many, Hk, H // Hk, d).permute(0, 2, 3, 1, 4).reshape(n, Hk, -1, d)
    p = (q @ k.transpose(2, 3)).mul_(d ** -0.5).reshape(n, Hk, H // Hk, many, -1)
    pos = (lens - new + i).unsqueeze(2)
    x = j.unsqueeze(1)
    sees = there.unsqueeze(1) & (x <= pos) & ((pos - x < W) | (x < S))
    p.masked_fill_(~sees[:, None, None], -math.inf)
    top = p.amax(dim=4, keepdim=True).clamp_min(-3e38)
    p.sub_(top).exp_()
    total = p.sum(dim=4, keepdim=True)
    o = (p.reshape(n, Hk, -1, p.shape[4]) @ v).reshape(n, Hk, H // Hk, many, d) / total
    lse = (top + total.log()).squeeze(4)
    real = i < new
    o = o.permute(0, 3, 1, 2, 4).reshape(n, many, H, d)[real]
    return {"o": o.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2).reshape(n, many, H)[real]}


def _angles(positions, inv_freq):
    """cos and sin of position * frequency, the angle in 64 bits: a far position's has no bits left in 32."""
    a = positions.double().unsqueeze(1) * inv_freq.double()
    return a.cos().float().unsqueeze(1), a.sin().float().unsqueeze(1)


def _turned(x, cos, sin, interleaved):
    """Pairs of the last axis turned by their angles; x [T, heads, dr] fp32."""
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    u, w = a * cos - b * sin, b * cos + a * sin
    return torch.stack([u, w], dim=-1).flatten(-2) if interleaved else torch.cat([u, w], dim=-1)


def _part_turned(x, start, dr, cos, sin, interleaved):
    return torch.cat([x[..., :start], _turned(x[..., start:start + dr], cos, sin, interleaved), x[..., start + dr:]],
                     dim=-1)


def _append(s):
    c = s["case"]
    Hk, d, dr, page = c["Hk"], c["d"], c["dr"], c["page"]
    k, v = s["kv"][:, :Hk], s["kv"][:, Hk:]
    if own:
        import gated_delta_rule_prefill_amd as kda
        out = kda.kv_append(s["k_cache"], s["v_cache"], k, v, s["block_table"], s["seq_lens"],
                            cu_seqlens=s["cu_seqlens"], norm_weight=s["norm_weight"], eps=EPS, inv_freq=s["inv_freq"],
                            interleaved=c["interleaved"], k_out=c["outs"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "k": out}
    cu = s["cu_seqlens"].long()
    t = torch.arange(k.shape[0], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    position = s["seq_lens"].long()[seq] - (cu[seq + 1] - t)
    x = k.float()
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + EPS) * s["norm_weight"]
    if dr:
        x = _part_turned(x, 0, dr, *_angles(position, s["inv_freq"]), c["interleaved"])
    x = x.to(k.dtype)
    rows = s["block_table"][seq, position // page].long() * page + position % page
    s["k_cache"].view(-1, Hk, d)[rows] = x
    s["v_cache"].view(-1, Hk, d)[rows] = v
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "k": x if c["outs"] else None}


def _norm(s):
    c = s["case"]
    H, Hk, start, dr = c["H"], c["Hk"], c["start"], c["dr"]
    q, k = s["qkv"][:, :H], s["qkv"][:, H:H + Hk]
    if own:
        import gated_delta_rule_prefill_amd as kda
        args = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], positions=s["positions"], inv_freq=s["inv_freq"],
                    start=start, interleaved=c["interleaved"], eps=EPS)
        yq, yk = kda.qk_norm_rotary(q, k, **args)
        if not c["train"]:
            return {"q": yq, "k": yk}
        g = kda.qk_norm_rotary_backward(q, k, s["dq"], s["dk"], **args)
        return {"q": yq, "k": yk, "dq": g["dq"], "dk": g["dk"], "dq_weight": g["dq_weight"],
                "dk_weight": g["dk_weight"]}
    cos, sin = _angles(s["positions"], s["inv_freq"])
    out = {}
    for name, x, w in (("q", q, s["q_weight"]), ("k", k, s["k_weight"])):
        x = x.float()
        r = torch.rsqrt((x * x).mean(dim=2, keepdim=True) + EPS)
        out[name] = _part_turned(x * r * w, start, dr, cos, sin, c["interleaved"]).to(q.dtype)
        if c["train"]:
            g = _part_turned(s["d" + name].float(), start, dr, cos, -sin, c["interleaved"])   # turned back
            n = x * r
            out["d" + name + "_weight"] = (g * n).sum(dim=(0, 1))
            h = g * w
            out["d" + name] = (r * (h - n * (h * n).mean(dim=2, keepdim=True))).to(q.dtype)
    return out


# -- what a pass cannot do without --------------------------------------------

def _seen(n, m, W, S):
    """Visible pairs of one sequence of n queries and m >= n keys."""
    total = 0
    for p in range(m - n, m):
        lo = max(0, p - W + 1)
        total += p - lo + 1 + min(S, lo)
    return total


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    d, Hk = case["d"], case["Hk"]
    if case["kind"] == "norm":
        n = case["T"] * (case["H"] + Hk)
        return {"bytes": n * d * es * (5 if case["train"] else 2) + 4 * case["T"],
                "flops": n * (d * (18 if case["train"] else 4) + case["dr"] * (6 if case["train"] else 3))}
    lens = _ints(case["lens"])
    if case["kind"] in ("attn", "train"):
        H, W, S = case["H"], case["window"], case["sinks"]
        T, Tk = sum(lens), sum(lens) + len(lens) * case["prefix"]
        pairs = H * sum(_seen(n, n + case["prefix"], W, S) for n in lens)
        q, kv = T * H * d, Tk * 2 * Hk * d
        if case["kind"] == "attn":
            return {"bytes": (2 * q + kv) * es + 4 * T * H, "flops": 4 * pairs * d}
        # inputs, the output and its gradient, the gradients; four products of the backward pass beside two of the forward
        return {"bytes": (4 * q + 2 * kv) * es, "flops": 12 * pairs * d}
    new = _ints(case["new"])
    T = sum(new)
    if case["kind"] == "decode":
        H, W, S = case["H"], case["window"], case["sinks"]
        pairs = H * sum(_seen(n, m, W, S) for n, m in zip(new, lens))
        rows = 0
        for n, m in zip(new, lens):                       # cached rows that some new token sees
            lo = max(0, m - n - W + 1)
            rows += m - lo + min(S, lo)
        return {"bytes": (rows * 2 * Hk * d + 2 * T * H * d) * es + 4 * T * H, "flops": 4 * pairs * d}
    moved = (5 if case["outs"] else 4) * T * Hk * d
    return {"bytes": moved * es, "flops": T * Hk * (4 * d + 3 * case["dr"])}


# -- the definition in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attention, "train": _exact_attention, "decode": _exact_decode, "append": _exact_append,
            "norm": _exact_norm}[case["kind"]](case, s)


def _exact_heads(q, ks, vs, p, W, S, scale):
    """One query head: weights, output and log sum; p the queries' positions, keys from `lo` on and the first ones."""
    j = torch.arange(ks.shape[0], device="cuda")[None]
    dist = p[:, None] - j
    hidden = (dist < 0) | ((dist >= W) & (j >= S))
    z = torch.mm(q, ks.t().contiguous()) * scale
    z[hidden] = -math.inf
    total = torch.logsumexp(z, dim=1)
    w = torch.exp(z - total[:, None])
    return w, torch.mm(w, vs), total


def _exact_attention(case, s):
    """Head by head, sequence by sequence, 4,096 queries at a time against the keys up to the last one they see; keys
    before the window of the first of them, sinks aside, are cut off."""
    H, Hk, d, W, S = case["H"], case["Hk"], case["d"], case["window"], case["sinks"]
    train = case["kind"] == "train"
    T, Tk = s["q"].shape[0], s["kv"].shape[0]
    f64 = dict(dtype=torch.float64, device="cuda")
    o, lse, dq = torch.zeros(T, H, d, **f64), torch.zeros(T, H, **f64), torch.zeros(T, H, d, **f64)
    dk, dv = torch.zeros(Tk, Hk, d, **f64), torch.zeros(Tk, Hk, d, **f64)
    cu_q, cu_k = _offsets(s["lens"]), _offsets(s["lens_k"])
    for x, (n, m) in enumerate(zip(s["lens"], s["lens_k"])):
        for i in range(0, n, 4096):
            e = min(n, i + 4096)
            hi, cut = m - n + e, max(0, m - n + i - W + 1 - S)   # keys S .. S + cut - 1 are seen by none of these
            keys = torch.cat([torch.arange(0, min(S, hi)), torch.arange(min(S, hi) + cut, hi)]).cuda() if cut else \
                torch.arange(0, hi, device="cuda")
            p = torch.arange(i, e, device="cuda") + (m - n)
            p = p - cut                                      # positions and keys behind the cut move up together
            rows = slice(cu_q[x] + i, cu_q[x] + e)
            for h in range(H):
                kh = h // (H // Hk)
                ks, vs = s["kv"][cu_k[x] + keys, kh].double(), s["kv"][cu_k[x] + keys, Hk + kh].double()
                q = s["q"][rows, h].double()
                w, o[rows, h], lse[rows, h] = _exact_heads(q, ks, vs, p, W, S, d ** -0.5)
                if train:
                    g = s["d_o"][rows, h].double()
                    dw = torch.mm(g, vs.t().contiguous())
                    dz = w * (dw - (w * dw).sum(dim=1)[:, None]) * d ** -0.5
                    dq[rows, h] = torch.mm(dz, ks)
                    dk[cu_k[x] + keys, kh] += torch.mm(dz.t().contiguous(), q)
                    dv[cu_k[x] + keys, kh] += torch.mm(w.t().contiguous(), g)
    return {"o": o, "dq": dq, "dk": dk, "dv": dv} if train else {"o": o, "lse": lse}


def _exact_decode(case, s):
    """Sequence by sequence over its own rows of the pool."""
    T, H, d = s["q"].shape
    Hk, W, S, page = case["Hk"], case["window"], case["sinks"], case["page"]
    o = torch.zeros(T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    t = 0
    for x, (m, n) in enumerate(zip(s["lens"], s["new"])):
        seen = torch.zeros(m, dtype=torch.bool)
        seen[:S] = True
        seen[max(0, m - n - W + 1):] = True
        j = seen.nonzero().flatten().cuda()
        place = s["block_table"][x].long()[torch.div(j, page, rounding_mode="floor")]
        k, v = (s[name][place, j % page].double().transpose(0, 1).contiguous() for name in ("k_cache", "v_cache"))
        q = s["q"][t:t + n].double().reshape(n, Hk, H // Hk, d).transpose(0, 1).reshape(Hk, n * (H // Hk), d)
        z = torch.bmm(q, k.transpose(1, 2).contiguous()) * d ** -0.5
        pos = torch.arange(m - n, m, device="cuda").repeat_interleave(H // Hk)[:, None]
        z.masked_fill_((j > pos) | ((j <= pos - W) & (j >= S)), -math.inf)
        total = torch.logsumexp(z, dim=2)
        y = torch.bmm(torch.exp(z - total[:, :, None]), v)
        o[t:t + n] = y.reshape(Hk, n, H // Hk, d).transpose(0, 1).reshape(n, H, d)
        lse[t:t + n] = total.reshape(Hk, n, H // Hk).transpose(0, 1).reshape(n, H)
        t += n
    return {"o": o, "lse": lse}


def _exact_turn(x, positions, inv_freq, interleaved, sign):
    """Pairs as complex numbers times e^(i sign angle); x [T, heads, dr]."""
    h = x.shape[-1] // 2
    z = torch.complex(x[..., 0::2], x[..., 1::2]) if interleaved else torch.complex(x[..., :h], x[..., h:])
    a = (sign * positions.double()[:, None] * inv_freq.double()[None])[:, None]
    z = z * torch.polar(torch.ones_like(a), a)
    y = torch.empty_like(x)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = z.real, z.imag
    else:
        y[..., :h], y[..., h:] = z.real, z.imag
    return y


def _exact_append(case, s):
    Hk, dr, page = case["Hk"], case["dr"], case["page"]
    k = s["kv"][:, :Hk].double()
    if case["norm"]:
        k = k / torch.sqrt(k.square().sum(dim=2, keepdim=True) / case["d"] + EPS) * s["norm_weight"].double()
    place, seq = [], []
    for i, (m, n) in enumerate(zip(s["lens"], s["new"])):
        place += range(m - n, m)
        seq += [i] * n
    place, seq = torch.tensor(place, device="cuda"), torch.tensor(seq, device="cuda")
    if dr:
        k[..., :dr] = _exact_turn(k[..., :dr].clone(), place, s["inv_freq"], case["interleaved"], 1.0)
    pages = s["block_table"][seq, torch.div(place, page, rounding_mode="floor")].long()
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc[pages, place % page] = k
    vc[pages, place % page] = s["kv"][:, Hk:].double()
    return {"k_cache": kc, "v_cache": vc, "k": k if case["outs"] else None}


def _exact_norm(case, s):
    """y = R(n w), n = x / |x|; the gradient of x from the Jacobian of x / |x| applied to R^T dy w."""
    H, Hk, d, a, b = case["H"], case["Hk"], case["d"], case["start"], case["start"] + case["dr"]
    out = {}
    for name, x, w in (("q", s["qkv"][:, :H], s["q_weight"]), ("k", s["qkv"][:, H:H + Hk], s["k_weight"])):
        x, w = x.double(), w.double()
        size = torch.sqrt(x.square().sum(dim=2, keepdim=True) / d + EPS)
        y = x / size * w
        y[..., a:b] = _exact_turn(y[..., a:b].clone(), s["positions"], s["inv_freq"], case["interleaved"], 1.0)
        out[name] = y
        if case["train"]:
            g = s["d" + name].double()
            g[..., a:b] = _exact_turn(g[..., a:b].clone(), s["positions"], s["inv_freq"], case["interleaved"], -1.0)
            out["d" + name + "_weight"] = torch.einsum("thd,thd->d", g, x / size)
            g *= w
            out["d" + name] = g / size - x * (x * g).sum(dim=2, keepdim=True) / (d * size ** 3)
    return out
