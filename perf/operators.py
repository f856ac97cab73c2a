"""Measurement cases of the latent-attention operators: what they compute in
plain torch operations, and the calls a program makes of the library instead.

A full-attention layer beside the KDA layers keeps one latent vector per token
(``dl`` channels, RMS-normalised) and one rotary key part shared by the heads
(``dr`` channels).  Four operators serve it:

  attention  the expanded form over packed sequences: per-head keys and values
             expanded from the latents, causal, forward, and as a training step
             with the gradients of q, k, v and the shared rotary key part;
  decode     the absorbed form over a paged cache of latents: queries already
             multiplied into the latent space, one or more new tokens per
             sequence, output in the latent space;
  append     a token's latent (normalised) and rotary key part (rotated) written
             to its place in the paged cache;
  rotary     rotary positions on part of a head, both layouts, with
             frequencies scaled for long contexts, and the inverse rotation.

``own`` selects the library's calls; otherwise ``run`` computes the plain form
in 32 bits, rounded once at the end.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


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
        dict(name="attn-f32-ragged", kind="attn", dtype="f32", H=4, d=64, dr=64, lens="1,130,17,64,77,5",
             prefix=0, causal=True),
        # one long prompt of a full-size layer: 16,384 tokens, 32 heads of 128 + 64 channels
        dict(name="attn-bf16-16384", kind="attn", dtype="bf16", H=32, d=128, dr=64, lens="16384", prefix=0,
             causal=True),
        # a small fp32 training step over ragged documents (gradient checks, small models)
        dict(name="train-f32-ragged", kind="train", dtype="f32", H=4, d=128, dr=64, lens="300,1,65,129",
             prefix=0, causal=True),
        # a training step of a full-size layer over 16 packed documents of 256 to 4,096 tokens
        dict(name="train-bf16-packed16", kind="train", dtype="bf16", H=32, d=128, dr=64,
             lens=_text(_uniform(3, 16, 256, 4096)), prefix=0, causal=True),
        # one sequence alone, 65,536 tokens in the cache, one new token: the latency of long-context decoding
        dict(name="decode-one-65536", kind="decode", dtype="bf16", H=32, dl=512, dr=64, page=64, lens="65536",
             new="1"),
        # the serving batch: 256 sequences of 256 to 8,192 tokens, one new token each
        dict(name="decode-256", kind="decode", dtype="bf16", H=32, dl=512, dr=64, page=64,
             lens=_text(_uniform(7, 256, 256, 8192)), new=_text([1] * 256)),
        # chunks of 128 new tokens of 16 prompts over their cached prefixes (chunked prefill, resumed prefixes)
        dict(name="decode-chunk-16x128", kind="decode", dtype="bf16", H=32, dl=512, dr=64, page=64,
             lens=_text(_uniform(6, 16, 1024, 4096)), new=_text([128] * 16)),
        # a small fp32 cache: short sequences, odd page size, one to three new tokens (speculative checks)
        dict(name="decode-f32-small", kind="decode", dtype="f32", H=8, dl=256, dr=64, page=16, lens="200,1,77,333",
             new="1,1,3,2"),
        # the cache write of one serving step: 256 sequences, one token each
        dict(name="append-step-256", kind="append", dtype="bf16", dl=512, dr=64, page=64,
             lens=_text(_uniform(7, 256, 256, 8192)), new=_text([1] * 256), interleaved=True, outs=False),
        # the cache write of 16 whole prompts, which also keeps the normalised latents for their expansion
        dict(name="append-prompts-16", kind="append", dtype="bf16", dl=512, dr=64, page=64,
             lens=_text(_uniform(3, 16, 256, 4096)), new=_text(_uniform(3, 16, 256, 4096)), interleaved=False,
             outs=True),
        # the query rotation of one serving step: 256 tokens, the last 64 of 192 channels, far positions
        dict(name="rotary-step-256", kind="rotary", dtype="bf16", T=256, H=32, d=192, start=128, dr=64,
             interleaved=True, far=1000000, scaled=True, inverse=False),
        # the query rotation of a 65,536-token prompt; inverse as the gradient takes it
        dict(name="rotary-65536", kind="rotary", dtype="bf16", T=65536, H=32, d=192, start=128, dr=64,
             interleaved=False, far=65536, scaled=True, inverse=True),
    ]


def _draw_attention(rng):
    train = rng.random() < 0.5
    f32 = rng.random() < 0.3
    H = rng.choice([1, 2, 3, 5, 8, 16, 32])
    d, dr = rng.choice([64, 128]), rng.choice([0, 64])
    causal = rng.random() < 0.85
    total = _log_int(rng, 16, 2048 if f32 else 16384 // (2 if train else 1) // (1 if causal else 2))
    n = min(total, _log_int(rng, 1, 24))
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    # now and then keys longer than the queries: new tokens after an expanded prefix
    prefix = _log_int(rng, 1, 1024) if rng.random() < 0.25 else 0
    return dict(kind="train" if train else "attn", dtype="f32" if f32 else "bf16", H=H, d=d, dr=dr,
                lens=_text(lens), prefix=prefix, causal=causal)


def _draw_decode(rng):
    f32 = rng.random() < 0.25
    H = rng.choice([1, 5, 8, 16, 32, 64, 128])
    n = _log_int(rng, 1, 32 if f32 else 256)
    top = max(2, min(65536, (40000 if f32 else 800000) // n))
    hi = _log_int(rng, 1, top)
    lens = [rng.randint(max(1, hi // 8), hi) for _ in range(n)]
    if rng.random() < 0.5:
        new = [1] * n
    else:
        most = _log_int(rng, 1, max(1, min(256, int(6e7 // (H * n * max(lens))) if H * n * max(lens) < 6e7 else 1)))
        new = [rng.randint(1, min(most, x)) for x in lens]
    return dict(kind="decode", dtype="f32" if f32 else "bf16", H=H, dl=rng.choice([256, 512]),
                dr=rng.choice([0, 64]), page=rng.choice([1, 16, 48, 64, 128]), lens=_text(lens), new=_text(new))


def _draw_append(rng):
    n = _log_int(rng, 1, 256)
    hi = _log_int(rng, 1, max(1, 60000 // n))
    new = [rng.randint(1, hi) for _ in range(n)] if rng.random() < 0.5 else [1] * n
    lens = [x + _log_int(rng, 1, 4096) - 1 for x in new]
    return dict(kind="append", dtype=rng.choice(["bf16", "bf16", "f32"]), dl=rng.choice([256, 512]),
                dr=rng.choice([0, 64]), page=rng.choice([1, 16, 48, 64, 128]), lens=_text(lens), new=_text(new),
                interleaved=rng.random() < 0.5, outs=rng.random() < 0.5)


def _draw_rotary(rng):
    dr = rng.choice([32, 64, 96, 128])
    start = rng.choice([0, 64, 128])
    return dict(kind="rotary", dtype=rng.choice(["bf16", "bf16", "f32"]), T=_log_int(rng, 1, 30000),
                H=rng.choice([1, 3, 8, 32]), d=start + dr + rng.choice([0, 0, 32]), start=start, dr=dr,
                interleaved=rng.random() < 0.5, far=_log_int(rng, 1, 4000000), scaled=rng.random() < 0.5,
                inverse=rng.random() < 0.5)


def draw(rng):
    return rng.choice([_draw_attention, _draw_attention, _draw_decode, _draw_decode, _draw_append,
                       _draw_rotary])(rng)


# -- inputs --------------------------------------------------------------------

def _inv_freq(dr, scaled):
    """Rotary frequencies base^(-2i/dr), base 10,000; scaled: the slow ones
    divided by 32 with a ramp between the fast and the slow, and the amplitude
    0.1 ln 32 + 1 that goes with it."""
    f = 10000.0 ** (-torch.arange(0, dr, 2, dtype=torch.float64) / dr)
    if not scaled:
        return f.float().cuda(), 1.0
    turns = 4096.0 * f / (2.0 * math.pi)     # full turns over the trained context
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return (f * keep + f / 32.0 * (1.0 - keep)).float().cuda(), 0.1 * math.log(32.0) + 1.0


def _offsets(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return at


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

    s = dict(case=case)
    if case["kind"] == "rotary":
        s["x"] = normal(case["T"], case["H"], case["d"])
        s["positions"] = torch.randint(0, case["far"], (case["T"],), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"], s["mscale"] = _inv_freq(case["dr"], case["scaled"])
        return s
    lens = _ints(case["lens"])
    n = len(lens)
    if case["kind"] in ("attn", "train"):
        H, d, dr = case["H"], case["d"], case["dr"]
        lens_k = [x + case["prefix"] for x in lens]
        T, Tk = sum(lens), sum(lens_k)
        # queries of unequal sharpness from head to head, as trained heads have
        sharp = 0.5 + 1.5 * torch.rand(H, 1, generator=g, device="cuda")
        s["q"] = (torch.randn(T, H, d + dr, generator=g, device="cuda") * sharp).to(dt)
        s["kv"] = normal(Tk, H, 2 * d)                    # what the expansion product leaves: keys, then values
        s["k_pe"] = normal(Tk, dr) if dr else None
        s["lens"], s["lens_k"] = lens, lens_k
        s["cu_q"] = torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda")
        s["cu_k"] = torch.tensor(_offsets(lens_k), dtype=torch.int32, device="cuda") if case["prefix"] else s["cu_q"]
        s["scale"] = 1.0 / math.sqrt(d + dr)
        if case["kind"] == "train":
            s["d_o"] = normal(T, H, d)
        return s
    new = _ints(case["new"])
    dl, dr, page = case["dl"], case["dr"], case["page"]
    T = sum(new)
    used = [-(-x // page) for x in lens]
    pages = sum(used) + sum(used) // 8 + 1                # a pool with some pages free
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, max(used)), -1, dtype=torch.int32)
    at = _offsets(used)
    place = torch.cat([torch.full((u,), i, dtype=torch.int64) for i, u in enumerate(used)])
    column = torch.cat([torch.arange(u) for u in used])
    table = table.cuda()
    table[place.cuda(), column.cuda()] = order[:at[-1]]
    s["block_table"] = table
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu_seqlens"] = torch.tensor(_offsets(new), dtype=torch.int32, device="cuda")
    s["lens"], s["new"] = lens, new
    s["cache"] = torch.empty(pages, page, dl + dr, dtype=dt, device="cuda")
    for a in range(0, pages, max(1, (1 << 16) // page)):  # filled in pieces: the fp32 draw of a large pool is as large again
        b = min(pages, a + max(1, (1 << 16) // page))
        s["cache"][a:b] = normal(b - a, page, dl + dr)
    if case["kind"] == "decode":
        # absorbed queries: their scores have a spread of a few units
        s["q"] = normal(T, case["H"], dl + dr, scale=2.0 / math.sqrt(dl + dr) * math.sqrt(192.0))
        s["scale"] = 1.0 / math.sqrt(192.0)               # of the heads before absorption
        return s
    s["c"] = normal(T, dl + dr)                           # the down projection's output: latent, then rotary key part
    s["norm_weight"] = 1.0 + 0.1 * torch.randn(dl, generator=g, device="cuda")
    s["inv_freq"], s["mscale"] = _inv_freq(dr, True) if dr else (None, 1.0)
    return s


# -- one pass --------------------------------------------------------------------

def run(state):
    return {"attn": _attention, "train": _train, "decode": _decode, "append": _append,
            "rotary": _rotary}[state["case"]["kind"]](state)


def _split(s):
    d = s["case"]["d"]
    return s["kv"][..., :d], s["kv"][..., d:]


def _attention(s):
    k, v = _split(s)
    if own:
        import gated_delta_rule_prefill_amd as kda
        o, lse = kda.latent_attention(s["q"], k, v, k_pe=s["k_pe"], cu_seqlens=s["cu_q"], cu_seqlens_k=s["cu_k"],
                                      causal=s["case"]["causal"], scale=s["scale"])
        return {"o": o, "lse": lse}
    T, H, d = s["q"].shape[0], s["case"]["H"], s["case"]["d"]
    o = torch.empty(T, H, d, dtype=s["q"].dtype, device="cuda")
    lse = torch.empty(T, H, device="cuda")
    a = b = 0
    for n, m in zip(s["lens"], s["lens_k"]):              # a sequence's scores at a time
        if n:
            qs, ks, vs = _heads(s, k, v, a, n, b, m)
            p, lse[a:a + n] = _probabilities(qs, ks, s["scale"], s["case"]["causal"])
            o[a:a + n] = (p @ vs).transpose(0, 1).to(o.dtype)
        a, b = a + n, b + m
    return {"o": o, "lse": lse}


def _heads(s, k, v, a, n, b, m):
    """A sequence's queries, whole keys and values, fp32, heads first."""
    qs = s["q"][a:a + n].float().transpose(0, 1)
    ks = k[b:b + m].float()
    if s["k_pe"] is not None:
        ks = torch.cat([ks, s["k_pe"][b:b + m].float().unsqueeze(1).expand(m, ks.shape[1], -1)], dim=2)
    return qs, ks.transpose(0, 1), v[b:b + m].float().transpose(0, 1)


def _probabilities(qs, ks, scale, causal):
    """softmax(scale q k^T) with row i seeing the keys up to i + (m - n), and the log of its sum."""
    n, m = qs.shape[1], ks.shape[1]
    p = qs @ ks.transpose(1, 2)
    p.mul_(scale)
    if causal:
        i = torch.arange(n, device=p.device).unsqueeze(1)
        p.masked_fill_(torch.arange(m, device=p.device) > i + (m - n), -math.inf)
    top = p.amax(dim=2, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(dim=2, keepdim=True)
    p.div_(total)
    return p, (top + total.log()).squeeze(2).transpose(0, 1)


def _train(s):
    k, v = _split(s)
    dr = s["case"]["dr"]
    if own:
        import gated_delta_rule_prefill_amd as kda
        args = dict(k_pe=s["k_pe"], cu_seqlens=s["cu_q"], cu_seqlens_k=s["cu_k"], causal=s["case"]["causal"],
                    scale=s["scale"])
        o, lse = kda.latent_attention(s["q"], k, v, **args)
        g = kda.latent_attention_backward(s["q"], k, v, o, lse, s["d_o"], **args)
        return {"o": o, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"], "dk_pe": g["dk_pe"]}
    T, H, d = s["q"].shape[0], s["case"]["H"], s["case"]["d"]
    Tk, dt = s["kv"].shape[0], s["q"].dtype
    o = torch.empty(T, H, d, dtype=dt, device="cuda")
    dq = torch.empty_like(s["q"])
    dk, dv = (torch.zeros(Tk, H, d, dtype=dt, device="cuda") for _ in range(2))
    dk_pe = torch.zeros_like(s["k_pe"]) if dr else None
    a = b = 0
    for n, m in zip(s["lens"], s["lens_k"]):
        if n:
            qs, ks, vs = _heads(s, k, v, a, n, b, m)
            p, _ = _probabilities(qs, ks, s["scale"], s["case"]["causal"])
            os = p @ vs
            gs = s["d_o"][a:a + n].float().transpose(0, 1)
            dv[b:b + m] = (p.transpose(1, 2) @ gs).transpose(0, 1).to(dt)
            ds = gs @ vs.transpose(1, 2)
            ds.sub_((gs * os).sum(dim=2, keepdim=True)).mul_(p).mul_(s["scale"])
            dq[a:a + n] = (ds @ ks).transpose(0, 1).to(dt)
            dks = (ds.transpose(1, 2) @ qs).transpose(0, 1)
            dk[b:b + m] = dks[..., :d].to(dt)
            if dr:
                dk_pe[b:b + m] = dks[..., d:].sum(dim=1).to(dt)
            o[a:a + n] = os.transpose(0, 1).to(dt)
        a, b = a + n, b + m
    return {"o": o, "dq": dq, "dk": dk, "dv": dv, "dk_pe": dk_pe}


def _gathered(cache, table, most):
    """The first `most` cached tokens of every sequence, [N, most, width]."""
    page = cache.shape[1]
    j = torch.arange(most, device=cache.device)
    rows = table[:, j // page].long().clamp(min=0) * page + j % page
    return cache.reshape(-1, cache.shape[2])[rows]


def _padded_tokens(cu, most):
    """Index [N, most] of every sequence's new tokens, and which of them exist."""
    i = torch.arange(most, device=cu.device)
    at = cu[:-1].long().unsqueeze(1) + i
    there = at < cu[1:].long().unsqueeze(1)
    return torch.where(there, at, torch.zeros_like(at)), there


def _decode(s):
    c = s["case"]
    if own:
        import gated_delta_rule_prefill_amd as kda
        o, lse = kda.latent_decode(s["q"], s["cache"], s["block_table"], s["seq_lens"], latent_dim=c["dl"],
                                   scale=s["scale"], cu_seqlens=s["cu_seqlens"])
        return {"o": o, "lse": lse}
    T, H, D = s["q"].shape
    most, many, n = max(s["lens"]), max(s["new"]), len(s["lens"])
    kv = _gathered(s["cache"], s["block_table"], most).float()
    at, there = _padded_tokens(s["cu_seqlens"], many)
    q = s["q"].float()[at].reshape(n, many * H, D)
    p = (q @ kv.transpose(1, 2)).mul_(s["scale"]).reshape(n, many, H, most)
    new = (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).long()
    last = s["seq_lens"].long().unsqueeze(1) - new.unsqueeze(1) + torch.arange(many, device=q.device)
    j = torch.arange(most, device=q.device)
    p.masked_fill_((j > last.unsqueeze(2)).unsqueeze(2) | ~there[:, :, None, None], -math.inf)
    top = p.amax(dim=3, keepdim=True).clamp_min(-3e38)
    p.sub_(top).exp_()
    total = p.sum(dim=3, keepdim=True)
    # places past a sequence's end weigh nothing whatever the pool holds there
    kv = torch.where((j < s["seq_lens"].unsqueeze(1)).unsqueeze(2), kv, torch.zeros_like(kv))
    o = (p.reshape(n, many * H, most) @ kv[:, :, :c["dl"]]).reshape(n, many, H, c["dl"]) / total
    lse = (top + total.log()).squeeze(3)
    return {"o": o[there].to(s["q"].dtype), "lse": lse[there]}


def _angles(positions, inv_freq):
    """cos and sin of position * frequency, the angle in 64 bits: a far position's has no bits left in 32."""
    a = positions.double().unsqueeze(1) * inv_freq.double()
    return a.cos().float(), a.sin().float()


def _turned(x, cos, sin, interleaved):
    """Pairs of the last axis turned by their angles, fp32; cos and sin broadcast over the axes between."""
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    u, w = a * cos - b * sin, b * cos + a * sin
    return torch.stack([u, w], dim=-1).flatten(-2) if interleaved else torch.cat([u, w], dim=-1)


def _append(s):
    c = s["case"]
    dl, dr = c["dl"], c["dr"]
    latent, k_pe = s["c"][:, :dl], s["c"][:, dl:] if dr else None
    if own:
        import gated_delta_rule_prefill_amd as kda
        got = kda.latent_append(s["cache"], latent, s["block_table"], s["seq_lens"], k_pe=k_pe,
                                cu_seqlens=s["cu_seqlens"], norm_weight=s["norm_weight"], eps=1e-6,
                                inv_freq=s["inv_freq"], interleaved=c["interleaved"], mscale=s["mscale"],
                                c_out=c["outs"], k_pe_out=c["outs"] and dr > 0)
        return {"cache": s["cache"], "c": got[0], "k_pe": got[1]}
    T, page, dt = s["c"].shape[0], c["page"], s["c"].dtype
    cu = s["cu_seqlens"].long()
    t = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    position = s["seq_lens"].long()[seq] - (cu[seq + 1] - t)
    x = latent.float()
    x = (x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + 1e-6) * s["norm_weight"]).to(dt)
    if dr:
        cos, sin = _angles(position, s["inv_freq"])
        pe = (_turned(k_pe.float(), cos, sin, c["interleaved"]) * s["mscale"]).to(dt)
    rows = s["block_table"][seq, position // page].long() * page + position % page
    s["cache"].view(-1, dl + dr)[rows] = torch.cat([x, pe], dim=1) if dr else x
    return {"cache": s["cache"], "c": x if c["outs"] else None, "k_pe": pe if c["outs"] and dr else None}


def _rotary(s):
    c = s["case"]
    if own:
        import gated_delta_rule_prefill_amd as kda
        return {"y": kda.rotary(s["x"], s["positions"], s["inv_freq"], start=c["start"], interleaved=c["interleaved"],
                                mscale=s["mscale"], inverse=c["inverse"])}
    cos, sin = _angles(s["positions"], s["inv_freq"])
    sin = -sin if c["inverse"] else sin
    a, b = c["start"], c["start"] + c["dr"]
    y = _turned(s["x"][..., a:b].float(), cos.unsqueeze(1), sin.unsqueeze(1), c["interleaved"]) * s["mscale"]
    out = s["x"].clone()
    out[..., a:b] = y.to(out.dtype)
    return {"y": out}


# -- what a pass cannot do without --------------------------------------------

def _visible(n, m, causal):
    """Query-key pairs of one sequence of n queries and m >= n keys."""
    return n * m - n * (n - 1) // 2 if causal else n * m


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "rotary":
        n = case["T"] * case["H"]
        return {"bytes": 2 * n * case["d"] * es + 4 * case["T"], "flops": 3 * n * case["dr"]}
    lens = _ints(case["lens"])
    if case["kind"] in ("attn", "train"):
        H, d, dr = case["H"], case["d"], case["dr"]
        T, Tk = sum(lens), sum(lens) + len(lens) * case["prefix"]
        pairs = H * sum(_visible(n, n + case["prefix"], case["causal"]) for n in lens)
        q, kv, o = T * H * (d + dr), Tk * (2 * H * d + dr), T * H * d
        if case["kind"] == "attn":
            return {"bytes": (q + kv + o) * es + 4 * T * H, "flops": 2 * pairs * (2 * d + dr)}
        # inputs, the output and its gradient, the gradients; four products of the backward pass beside two of the forward
        return {"bytes": (2 * q + 2 * kv + 2 * o) * es, "flops": 2 * pairs * 3 * (2 * d + dr)}
    new, dl, dr = _ints(case["new"]), case["dl"], case["dr"]
    T = sum(new)
    if case["kind"] == "decode":
        pairs = case["H"] * sum(_visible(n, m, True) for n, m in zip(new, lens))
        read = sum(lens) * (dl + dr) + T * case["H"] * (dl + dr)
        return {"bytes": (read + T * case["H"] * dl) * es + 4 * T * case["H"], "flops": 2 * pairs * (2 * dl + dr)}
    moved = 2 * T * (dl + dr) + (T * (dl + dr) if case["outs"] else 0)
    return {"bytes": moved * es + 4 * dl, "flops": T * (4 * dl + 3 * dr)}


# -- the definition in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attention, "train": _exact_attention, "decode": _exact_decode, "append": _exact_append,
            "rotary": _exact_rotary}[case["kind"]](case, s)


def _exact_attention(case, s):
    """Head by head and sequence by sequence: weights w_ij = exp(z_ij - log sum_j exp z_ij) over the visible j."""
    H, d, dr, train = case["H"], case["d"], case["dr"], case["kind"] == "train"
    T, Tk = s["q"].shape[0], s["kv"].shape[0]
    f64 = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(T, H, d, **f64), torch.zeros(T, H, **f64)
    dq, dk, dv = (torch.zeros(t, H, w, **f64) for t, w in ((T, d + dr), (Tk, d), (Tk, d)))
    dk_pe = torch.zeros(Tk, dr, **f64)
    cu_q, cu_k = _offsets(s["lens"]), _offsets(s["lens_k"])
    for i, (n, m) in enumerate(zip(s["lens"], s["lens_k"])):
        if not n:
            continue
        qr, kr = slice(cu_q[i], cu_q[i + 1]), slice(cu_k[i], cu_k[i + 1])
        hidden = None
        if case["causal"]:
            hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1)
        for h in range(H):
            q, v = s["q"][qr, h].double(), s["kv"][kr, h, d:].double()
            k = s["kv"][kr, h, :d].double()
            if dr:
                k = torch.hstack([k, s["k_pe"][kr].double()])
            z = torch.mm(q, k.t().contiguous()) * s["scale"]
            if hidden is not None:
                z[hidden] = -math.inf
            total = torch.logsumexp(z, dim=1)
            w = torch.exp(z - total[:, None])
            o[qr, h], lse[qr, h] = torch.mm(w, v), total
            if train:
                g = s["d_o"][qr, h].double()
                dv[kr, h] = torch.mm(w.t().contiguous(), g)
                dw = torch.mm(g, v.t().contiguous())
                dz = w * (dw - (w * dw).sum(dim=1)[:, None]) * s["scale"]
                dq[qr, h] = torch.mm(dz, k)
                dkh = torch.mm(dz.t().contiguous(), q)
                dk[kr, h] = dkh[:, :d]
                dk_pe[kr] += dkh[:, d:]
    if train:
        return {"o": o, "dq": dq, "dk": dk, "dv": dv, "dk_pe": dk_pe if dr else None}
    return {"o": o, "lse": lse}


def _exact_decode(case, s):
    """Sequence by sequence over its own rows of the pool."""
    T, H, _ = s["q"].shape
    dl, page = case["dl"], case["page"]
    o = torch.zeros(T, H, dl, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    t = 0
    for i, (m, n) in enumerate(zip(s["lens"], s["new"])):
        pages = s["block_table"][i, :-(-m // page)].long()
        rows = s["cache"][pages].reshape(-1, s["cache"].shape[2])[:m].double()
        z = torch.mm(s["q"][t:t + n].double().reshape(n * H, -1), rows.t().contiguous()) * s["scale"]
        z = z.reshape(n, H, m)
        for u in range(n):
            z[u, :, m - n + u + 1:] = -math.inf
        total = torch.logsumexp(z, dim=2)
        w = torch.exp(z - total[:, :, None]).reshape(n * H, m)
        o[t:t + n] = torch.mm(w, rows[:, :dl].contiguous()).reshape(n, H, dl)
        lse[t:t + n] = total
        t += n
    return {"o": o, "lse": lse}


def _exact_turn(x, positions, inv_freq, interleaved, mscale, sign):
    """Pairs as complex numbers times mscale e^(i sign angle); x [T, ..., dr]."""
    h = x.shape[-1] // 2
    z = torch.complex(x[..., 0::2], x[..., 1::2]) if interleaved else torch.complex(x[..., :h], x[..., h:])
    a = sign * positions.double()[:, None] * inv_freq.double()[None]
    a = a.reshape(a.shape[0], *([1] * (x.dim() - 2)), h)
    z = z * torch.polar(torch.full_like(a, mscale), a)
    y = torch.empty_like(x)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = z.real, z.imag
    else:
        y[..., :h], y[..., h:] = z.real, z.imag
    return y


def _exact_append(case, s):
    dl, dr, page = case["dl"], case["dr"], case["page"]
    x = s["c"].double()
    c = x[:, :dl] / torch.sqrt(x[:, :dl].square().sum(dim=1, keepdim=True) / dl + 1e-6) * s["norm_weight"].double()
    place, seq = [], []
    for i, (m, n) in enumerate(zip(s["lens"], s["new"])):
        place += range(m - n, m)
        seq += [i] * n
    place, seq = torch.tensor(place, device="cuda"), torch.tensor(seq, device="cuda")
    pe = _exact_turn(x[:, dl:], place, s["inv_freq"], case["interleaved"], s["mscale"], 1.0) if dr else x[:, dl:]
    cache = s["cache"].double()
    pages = s["block_table"][seq, torch.div(place, page, rounding_mode="floor")].long()
    cache[pages, place % page] = torch.hstack([c, pe])
    return {"cache": cache, "c": c if case["outs"] else None, "k_pe": pe if case["outs"] and dr else None}


def _exact_rotary(case, s):
    y = s["x"].double()
    a, b = case["start"], case["start"] + case["dr"]
    y[..., a:b] = _exact_turn(y[..., a:b].clone(), s["positions"], s["inv_freq"], case["interleaved"], s["mscale"],
                              -1.0 if case["inverse"] else 1.0)
    return {"y": y}
