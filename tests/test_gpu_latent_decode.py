"""Absorbed latent attention over a paged cache, the cache's writes and rotary
positions against their definitions in float64, element by element."""
import math

import pytest
import torch

import latent_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def offsets(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def make(seed, dtype, H, dl, dr, page, lens, new, poison=True, behind=0):
    """A pool whose pages lie in random order; rows behind a sequence's end and
    free pages hold NaN (nothing of them may reach a result)."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-m // page) for m in lens]
    P = sum(used) + 3
    order = torch.randperm(P, generator=g)
    table = torch.full((len(lens), max(1, max(used))), -1, dtype=torch.int32)
    cache = torch.full((P, page, dl + dr), float("nan") if poison else 0.0)
    at = 0
    for s, (m, u) in enumerate(zip(lens, used)):
        pages = order[at:at + u]
        table[s, :u] = pages.int()
        rows = torch.randn(m, dl + dr, generator=g)
        for i, p in enumerate(pages):
            part = rows[i * page:(i + 1) * page]
            cache[p, :part.shape[0]] = part
        at += u
    T = sum(new) + behind
    q = torch.randn(T, H, dl + dr, generator=g) * 1.2
    return dict(q=q.to(DT[dtype]).cuda(), cache=cache.to(DT[dtype]).cuda(), table=table.cuda(),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), cu=offsets(new), scale=192 ** -0.5)


def run(x, dl, **kw):
    import gated_delta_rule_prefill_amd as kda
    kw.setdefault("cu_seqlens", x["cu"])
    return kda.latent_decode(x["q"], x["cache"], x["table"], x["seq_lens"], latent_dim=dl, scale=x["scale"], **kw)


def check(label, x, dl, lens, new, **kw):
    o, lse = run(x, dl, **kw)
    torch.cuda.synchronize()
    (wo, eo), (wl, el) = ref.decode(x["q"], x["cache"], x["table"], lens, new, dl, x["scale"])
    n = sum(new)
    ref.check(f"{label} o", o[:n], wo[:n], eo[:n])
    ref.check(f"{label} lse", lse[:n], wl[:n], el[:n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dl,dr", [(512, 64), (512, 0), (256, 64), (256, 0)])
@pytest.mark.parametrize("H", [1, 5, 32, 128])
def test_single_tokens(dtype, dl, dr, H):
    lens = [1, 64, 65, 0, 300, 17]
    x = make(31, dtype, H, dl, dr, 16, lens, [1] * 6)
    check(f"{dtype} {dl}+{dr} H={H}", x, dl, lens, [1] * 6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 7, 48, 64, 100, 128])
def test_page_sizes_and_several_tokens(dtype, page):
    lens, new = [40, 3, 200, 129, 64], [3, 3, 1, 0, 7]
    x = make(32, dtype, 8, 256, 64, page, lens, new)
    check(f"{dtype} page {page}", x, 256, lens, new)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunks_of_new_tokens(dtype):
    """Many rows per sequence; a whole prompt (no prefix); more new tokens than
    the cache is said to hold (rows that see nothing)."""
    lens, new = [260, 70, 10, 33], [65, 70, 14, 1]
    x = make(33, dtype, 8, 512, 64, 64, lens, new)
    check(f"{dtype} chunks", x, 512, lens, new)


def test_equal_rows():
    lens = [100, 40, 77]
    x = make(34, "bf16", 16, 512, 64, 64, lens, [2, 2, 2])
    check("equal rows", x, 512, lens, [2, 2, 2], cu_seqlens=None)


def test_one_long_sequence():
    """One sequence split over every workgroup, its parts joined."""
    lens = [20000]
    x = make(35, "bf16", 32, 512, 64, 64, lens, [1])
    check("20000 tokens", x, 512, lens, [1])


def test_mixed_lengths_over_workgroups():
    lens = [5000, 1, 0, 3, 9000, 64, 2000] + [30] * 40
    new = [1, 1, 1, 1, 2, 1, 1] + [1] * 40
    x = make(36, "bf16", 8, 256, 64, 64, lens, new)
    check("mixed", x, 256, lens, new)


@pytest.mark.parametrize("H", [4, 40])
def test_many_sequences(H):
    """More sequences than a workgroup has threads, and more row tiles than workgroups."""
    lens = [(13 * i) % 90 for i in range(1100)]
    new = [1 if i % 7 else 0 for i in range(1100)]
    x = make(37, "bf16", H, 256, 0, 16, lens, new)
    check(f"1100 sequences H={H}", x, 256, lens, new)


def test_bad_pages_and_lengths():
    """Pages outside the pool count as absent; a length beyond the table's room
    is clamped to it, a negative one to zero."""
    lens = [100, 100, 50, 64]
    x = make(38, "bf16", 8, 256, 64, 16, lens, [1] * 4)
    x["table"][0, 2] = -1
    x["table"][1, 0] = x["cache"].shape[0]
    x["table"][1, 6] = 2 ** 31 - 1
    x["table"][2, :] = -5
    check("bad pages", x, 256, lens, [1] * 4)
    x = make(39, "bf16", 8, 256, 64, 16, [112, 112], [1] * 2, poison=False)
    x["seq_lens"][0] = 2 ** 31 - 1
    x["seq_lens"][1] = -3
    check("bad lengths", x, 256, [2 ** 31 - 1, -3], [1] * 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,value", [(1, "nan"), (32, "inf")])
def test_hidden_rows_that_are_not_finite(dtype, H, value):
    """Of a chunk of new tokens, those before a row with NaN or Inf are clean."""
    lens, new, bad = [150, 90], [30, 5], 130
    x = make(44, dtype, H, 256, 64, 16, lens, new, poison=False)
    (wo, eo), (wl, el) = ref.decode(x["q"], x["cache"], x["table"], lens, new, 256, x["scale"])
    x["cache"][int(x["table"][0, bad // 16]), bad % 16, 7] = float(value)
    x["cache"][int(x["table"][0, 149 // 16]), 149 % 16, 300] = float(value)
    o, lse = run(x, 256)
    for part in (slice(0, bad - 120), slice(30, 35)):
        ref.check("clean rows o", o[part], wo[part], eo[part])
        ref.check("clean rows lse", lse[part], wl[part], el[part])
    assert torch.isnan(o[bad - 120:30].float()).any(dim=-1).all()


def test_rows_behind_the_last_sequence_are_left():
    lens, new = [100, 30], [1, 2]
    x = make(40, "bf16", 32, 512, 64, 64, lens, new, behind=5)
    x["q"][3:] = float("nan")
    out = torch.full((8, 32, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, 32), 7.0, device="cuda")
    check("padded", x, 512, lens, new, out=out, lse=lse)
    assert (out[3:] == 7.0).all() and (lse[3:] == 7.0).all()


def test_rows_past_32_bit_offsets():
    """A pool of more than 2^31 elements: the last pages are read at their place."""
    dl, dr, page = 512, 64, 64
    P = 2 ** 31 // (page * (dl + dr)) + 40
    cache = torch.zeros(P, page, dl + dr, dtype=torch.bfloat16, device="cuda")
    lens = [130]
    x = make(41, "bf16", 8, dl, dr, page, lens, [1])
    far = torch.tensor([P - 1, P - 7, P - 2], dtype=torch.int32)
    for i in range(3):
        cache[int(far[i])] = x["cache"][int(x["table"][0, i])].nan_to_num(0.0)
    x["cache"], x["table"] = cache, far[None].cuda()
    check("past 2^31", x, dl, lens, [1])


def test_strided_queries_and_same_result_twice():
    lens, new = [700, 90], [1, 3]
    x = make(42, "bf16", 16, 512, 64, 64, lens, new)
    o0, l0 = run(x, 512)
    o1, l1 = run(x, 512)
    assert torch.equal(o0, o1) and torch.equal(l0, l1)
    heads_first = x["q"].transpose(0, 1).contiguous().transpose(0, 1)
    x["q"] = heads_first
    o2, l2 = run(x, 512)
    assert torch.equal(o0, o2) and torch.equal(l0, l2)


def test_two_captured_calls_with_their_own_workspaces():
    """Two decode graphs over different lengths replayed in turn with eager
    calls between; lengths and pages change in place between replays."""
    lens, new = [900, 64, 5], [1, 1, 1]
    xs = [make(43 + i, "bf16", 32, 512, 64, 64, lens, new, poison=False) for i in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in xs:
            run(x, 512)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(x, 512))
        graphs.append(g)
    for step in range(4):
        for x in xs:
            x["seq_lens"].copy_(torch.tensor([900 - 100 * step, 64 - step, 5 - step], dtype=torch.int32))
        want = [run(x, 512) for x in xs]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


# -- append and rotary --------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dl,dr,page,interleaved", [(512, 64, 64, True), (512, 64, 16, False), (256, 0, 7, False),
                                                    (1024, 256, 5, True), (64, 8, 1, False), (448, 72, 64, True)])
def test_append(dtype, dl, dr, page, interleaved):
    import gated_delta_rule_prefill_amd as kda
    lens, new = [40, 3, 700, 2, 64, 9], [3, 3, 650, 0, 1, 1]
    x = make(51, dtype, 1, dl, dr, page, lens, new, poison=False)
    x["table"][5, :] = -1                         # a token without a page: its outputs are written, the cache is not
    before = x["cache"].clone()
    T, dt = sum(new), DT[dtype]
    g = torch.Generator().manual_seed(3)
    wide = (torch.randn(T, dl + dr, generator=g) * 2).to(dt).cuda()
    c, k_pe = wide[:, :dl], wide[:, dl:] if dr else None
    w = (1 + 0.2 * torch.randn(dl, generator=g)).cuda()
    f, amp = kda.rotary_frequencies(dr, factor=8.0, original_context=1024, device="cuda") if dr else (None, 1.0)
    co, po = kda.latent_append(x["cache"], c, x["table"], x["seq_lens"], k_pe=k_pe, cu_seqlens=x["cu"], norm_weight=w,
                               eps=1e-5, inv_freq=f, interleaved=interleaved, mscale=amp, c_out=True,
                               k_pe_out=dr > 0)
    torch.cuda.synchronize()
    cd = c.double().cpu()
    want_c = cd / torch.sqrt((cd * cd).mean(1, keepdim=True) + 1e-5) * w.double().cpu()
    pos = torch.cat([torch.arange(m - n, m) for m, n in zip(lens, new)])
    u = ref.U[dt] + 1e-6
    ref.check("append c", co, want_c, u * want_c.abs())
    if dr:
        want_p = ref.turned(k_pe, pos, f, interleaved, amp)
        size = ref.turned(k_pe.abs(), pos * 0, f, interleaved, amp)
        h = dr // 2
        pair = size[:, 0::2] + size[:, 1::2] if interleaved else size[:, :h] + size[:, h:]
        pair = pair.repeat_interleave(2, 1) if interleaved else torch.cat([pair, pair], 1)
        ref.check("append k_pe", po, want_p, ref.U[dt] * want_p.abs() + 1e-6 * pair)
    # the cache: the rows of the new tokens and nothing else
    expect = before.view(-1, dl + dr)
    t = 0
    for s, (m, n) in enumerate(zip(lens, new)):
        for j in range(m - n, m):
            p = int(x["table"][s, j // page])
            if p >= 0:
                expect[p * page + j % page] = torch.cat([co[t], po[t]]) if dr else co[t]
            t += 1
    assert torch.equal(x["cache"].view(-1, dl + dr), expect)


def test_append_plain_rows_and_padding():
    """No norm, no rotation; equal rows; packed rows behind the last sequence
    and tokens at negative positions stay out of the cache."""
    import gated_delta_rule_prefill_amd as kda
    x = make(52, "bf16", 1, 256, 64, 16, [20, 33], [2, 2], poison=False)
    c = torch.randn(4, 320, device="cuda").bfloat16()
    before = x["cache"].clone()
    kda.latent_append(x["cache"], c[:, :256], x["table"], x["seq_lens"], k_pe=c[:, 256:])
    for t, (s, j) in enumerate([(0, 18), (0, 19), (1, 31), (1, 32)]):
        p = int(x["table"][s, j // 16])
        before[p, j % 16] = c[t]
    assert torch.equal(x["cache"], before)
    x["seq_lens"].copy_(torch.tensor([1, 33], dtype=torch.int32))
    cu = torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")
    co = torch.full((6, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    c = torch.randn(6, 320, device="cuda").bfloat16()
    kda.latent_append(x["cache"], c[:, :256], x["table"], x["seq_lens"], k_pe=c[:, 256:], cu_seqlens=cu, c_out=co)
    p = int(x["table"][0, 0])
    before[p, 0] = c[2]
    before[int(x["table"][1, 2]), 0] = c[3]
    assert torch.equal(x["cache"], before)
    assert torch.equal(co[:4], c[:4, :256]) and (co[4:] == 7.0).all()


def test_append_many_sequences():
    """The search of a token's sequence over several probes, empty ones between."""
    import gated_delta_rule_prefill_amd as kda
    N = 5000
    new = [(i * i) % 3 for i in range(N)]
    T = sum(new)
    table = torch.arange(N, dtype=torch.int32, device="cuda")[:, None].contiguous()
    cache = torch.zeros(N, 4, 64, device="cuda")
    seq_lens = torch.tensor([n + 1 for n in new], dtype=torch.int32, device="cuda")
    c = torch.randn(T, 64, device="cuda")
    kda.latent_append(cache, c, table, seq_lens, cu_seqlens=offsets(new))
    want = torch.zeros(N, 4, 64)
    t, ch = 0, c.cpu()
    for s, n in enumerate(new):
        want[s, 1:1 + n] = ch[t:t + n]
        t += n
    assert torch.equal(cache.cpu(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,d,start,dr", [(1, 1, 64, 0, 64), (37, 3, 192, 128, 64), (5, 32, 160, 64, 96),
                                            (300, 2, 70, 3, 10), (9, 5, 33, 1, 2), (2, 1, 4096, 0, 4096),
                                            (1000, 1, 64, 0, 32)])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("inverse", [True, False])
def test_rotary(dtype, T, H, d, start, dr, interleaved, inverse):
    import gated_delta_rule_prefill_amd as kda
    g = torch.Generator().manual_seed(d + T)
    x = torch.randn(T, H, d, generator=g).to(DT[dtype]).cuda()
    pos = torch.randint(-5, 4000000, (T,), generator=g, dtype=torch.int32).cuda()
    pos[0] = 2 ** 31 - 1
    f, amp = kda.rotary_frequencies(dr, factor=32.0, original_context=4096, device="cuda")
    y = kda.rotary(x, pos, f, start=start, interleaved=interleaved, mscale=amp, inverse=inverse)
    part = slice(start, start + dr)
    want = ref.turned(x[..., part], pos, f, interleaved, amp, inverse)
    # the angle is off by 2^31 f 2^-52 turns at most (4e-7 rad) and the rest by
    # fp32 roundings of both products
    size = x[..., part].double().cpu().abs().amax(-1, keepdim=True).expand_as(want) * amp
    ref.check("rotary", y[..., part], want, ref.U[DT[dtype]] * want.abs() + 2e-6 * size)
    keep = torch.ones(d, dtype=torch.bool)
    keep[part] = False
    assert torch.equal(y[..., keep.cuda()], x[..., keep.cuda()])
    z = x.clone()
    assert kda.rotary(z, pos, f, start=start, interleaved=interleaved, mscale=amp, inverse=inverse, out=z) is z
    assert torch.equal(z, y)
    # strided in and out (heads first; channels inside a wider row)
    hf = x.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((T, H, d + 5), 7.0, dtype=x.dtype, device="cuda")
    kda.rotary(hf, pos, f, start=start, interleaved=interleaved, mscale=amp, inverse=inverse, out=wide[..., :d])
    assert torch.equal(wide[..., :d], y) and (wide[..., d:] == 7.0).all()


def test_rotary_gradient_is_the_inverse():
    """<R x, g> = <x, R^-1 g>, and R^-1 R x = amplitude^2 x."""
    import gated_delta_rule_prefill_amd as kda
    x, g = (torch.randn(50, 4, 96, device="cuda") for _ in range(2))
    pos = torch.randint(0, 100000, (50,), dtype=torch.int32, device="cuda")
    f, amp = kda.rotary_frequencies(64, factor=4.0, original_context=2048, device="cuda")
    kw = dict(start=32, interleaved=True, mscale=amp)
    a = (kda.rotary(x, pos, f, **kw).double() * g.double()).sum()
    b = (x.double() * kda.rotary(g, pos, f, inverse=True, **kw).double()).sum()
    # 50 * 4 * 96 products of size about 1, each side's values off by 2^-23
    assert abs(float(a - b)) <= 50 * 4 * 96 * 4 * 2.0 ** -23
    back = kda.rotary(kda.rotary(x, pos, f, **kw), pos, f, inverse=True, **kw)
    assert torch.allclose(back[..., 32:], amp * amp * x[..., 32:], rtol=0, atol=2e-5)


def test_a_layer_step_by_step():
    """The operators as a layer uses them: a prompt through the expanded form
    and the cache, then tokens one by one through the absorbed form over that
    cache, against the expanded form over the whole sequence.  fp32, so that
    both agree to the rounding of the expansion products (1e-4 of the norm)."""
    import gated_delta_rule_prefill_amd as kda
    g = torch.Generator().manual_seed(9)
    H, dn, dr, dl, page, n, m = 8, 128, 64, 256, 16, 75, 5
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    wk, wv = r(dl, H, dn) / dl ** 0.5, r(dl, H, dn) / dl ** 0.5
    down, q = r(n + m, dl + dr), r(n + m, H, dn + dr)
    w = 1 + 0.1 * r(dl)
    f, amp = kda.rotary_frequencies(dr, factor=4.0, original_context=64, device="cuda")
    pos = torch.arange(n + m, dtype=torch.int32, device="cuda")
    q = kda.rotary(q, pos, f, start=dn, interleaved=True, mscale=amp)
    pages = (n + m + page - 1) // page
    cache = torch.full((pages + 2, page, dl + dr), float("nan"), device="cuda")
    table = torch.randperm(pages + 2, generator=g)[:pages].int()[None].cuda()
    kw = dict(norm_weight=w, inv_freq=f, interleaved=True, mscale=amp)

    def append(a, b, **more):
        return kda.latent_append(cache, down[a:b, :dl], table, torch.tensor([b], dtype=torch.int32, device="cuda"),
                                 k_pe=down[a:b, dl:], **kw, **more)
    scale = (dn + dr) ** -0.5
    c, k_pe = append(0, n, c_out=True, k_pe_out=True)
    k, v = torch.einsum("tl,lhd->thd", c, wk), torch.einsum("tl,lhd->thd", c, wv)
    prompt, _ = kda.latent_attention(q[:n], k, v, k_pe=k_pe, scale=scale)
    rows = []
    for t in range(n, n + m):
        append(t, t + 1)
        qa = torch.cat([torch.einsum("thd,lhd->thl", q[t:t + 1, :, :dn], wk), q[t:t + 1, :, dn:]], dim=2)
        o, _ = kda.latent_decode(qa, cache, table, torch.tensor([t + 1], dtype=torch.int32, device="cuda"),
                                 latent_dim=dl, scale=scale)
        rows.append(torch.einsum("thl,lhd->thd", o, wv))
    torch.cuda.synchronize()
    got = torch.cat([prompt] + rows)
    cd = down[:, :dl].double().cpu()
    cd = cd / torch.sqrt((cd * cd).mean(1, keepdim=True) + 1e-6) * w.double().cpu()
    pe = ref.turned(down[:, dl:], pos, f, True, amp)
    kd = torch.einsum("tl,lhd->thd", cd, wk.double().cpu())
    vd = torch.einsum("tl,lhd->thd", cd, wv.double().cpu())
    want, _ = ref.attention(q, kd, vd, pe, [n + m], [n + m], True, scale)["o"]
    err = (got.double().cpu() - want).norm() / want.norm()
    print(f"[latent] layer: rel-L2 {float(err):.2e}", flush=True)
    assert err <= 1e-4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_offsets_outside_the_tokens(dtype):
    """Offsets before 0 and behind T are clamped: the same rows as with offsets
    of 0 and T, which decode reads."""
    import gated_delta_rule_prefill_amd as kda
    c = torch.randn(6, 320, device="cuda").to(DT[dtype])
    for cu in ([0, 2, 6], [-3, 2, 11]):
        x = make(53, dtype, 8, 256, 64, 16, [20, 33], [2, 4], poison=False)
        offs = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kda.latent_append(x["cache"], c[:, :256], x["table"], x["seq_lens"], k_pe=c[:, 256:], cu_seqlens=offs)
        rows = x["cache"].view(-1, 320)
        for t, (s, j) in enumerate([(0, 18), (0, 19), (1, 29), (1, 30), (1, 31), (1, 32)]):
            assert torch.equal(rows[int(x["table"][s, j // 16]) * 16 + j % 16], c[t]), (cu, t)
        for a, b in zip(run(x, 256), run(x, 256, cu_seqlens=offs)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 32])
def test_key_parts_of_minus_infinity(dtype, H):
    """A key part that makes a score -inf takes its key out, as by the formula,
    in tiles that all rows see and in those that some do not: k_pe is no value."""
    lens, new = [150, 90], [30, 5]
    x = make(45, dtype, H, 256, 64, 16, lens, new, poison=False)
    x["q"][..., 300] = x["q"][..., 300].abs() + 0.5
    for s, j in ((0, 3), (0, 70), (0, 125), (0, 149), (1, 88)):
        x["cache"][int(x["table"][s, j // 16]), j % 16, 300] = -math.inf
    check(f"key parts of -inf {dtype} H={H}", x, 256, lens, new)
