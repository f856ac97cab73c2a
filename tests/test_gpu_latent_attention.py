"""Expanded latent attention and its gradients against the definition in
float64, element by element (bounds in latent_reference.py)."""
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


def make(seed, dtype, H, d, dr, lens_q, lens_k, behind=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    T, Tk = sum(lens_q) + behind, sum(lens_k) + behind
    r = lambda *s: (torch.randn(*s, generator=g) * spread).to(DT[dtype]).cuda()  # noqa: E731
    kv = r(Tk, H, 2 * d)
    return dict(q=r(T, H, d + dr), k=kv[..., :d], v=kv[..., d:], k_pe=r(Tk, dr) if dr else None,
                d_o=r(T, H, d), scale=(d + dr) ** -0.5)


def both(x, lens_q, lens_k, causal, packed=True, **kw):
    import gated_delta_rule_prefill_amd as kda
    args = dict(k_pe=x["k_pe"], causal=causal, scale=x["scale"], **kw)
    if packed:
        args["cu_seqlens"] = offsets(lens_q)
        if lens_k != lens_q:
            args["cu_seqlens_k"] = offsets(lens_k)
    else:
        args["num_seqs"] = len(lens_q)
    o, lse = kda.latent_attention(x["q"], x["k"], x["v"], **args)
    grads = kda.latent_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], **args)
    torch.cuda.synchronize()
    return dict(o=o, lse=lse, **grads)


def check_all(label, x, got, lens_q, lens_k, causal):
    want = ref.attention(x["q"], x["k"], x["v"], x["k_pe"], lens_q, lens_k, causal, x["scale"], x["d_o"])
    T, Tk = sum(lens_q), sum(lens_k)
    for name, (value, bound) in want.items():
        n = T if name in ("o", "lse", "dq") else Tk
        ref.check(f"{label} {name}", got[name][:n], value[:n], bound[:n])


RAGGED = [1, 0, 63, 64, 65, 128, 129, 2, 200]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,dr", [(128, 64), (128, 0), (64, 64), (64, 0)])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_batch(dtype, d, dr, causal):
    x = make(11, dtype, 3, d, dr, RAGGED, RAGGED)
    check_all(f"ragged {dtype} {d}+{dr} causal={causal}", x, both(x, RAGGED, RAGGED, causal), RAGGED, RAGGED, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens_q,lens_k", [
    ([5, 1, 70, 0, 33], [40, 130, 70, 9, 300]),      # new tokens after a prefix; keys without queries
    ([70, 130, 3], [20, 129, 0]),                    # rows that see no key
])
@pytest.mark.parametrize("causal", [True, False])
def test_unequal_lengths(dtype, lens_q, lens_k, causal):
    x = make(12, dtype, 8, 128, 64, lens_q, lens_k)
    check_all(f"unequal {dtype} {lens_q} {lens_k} causal={causal}", x, both(x, lens_q, lens_k, causal), lens_q,
              lens_k, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_rows_and_one_token(dtype):
    for lens in ([1], [97, 97, 97], [256, 256]):
        x = make(13, dtype, 4, 64, 64, lens, lens)
        check_all(f"rows {dtype} {lens}", x, both(x, lens, lens, True, packed=False), lens, lens, True)


def test_longer_sequence_and_sharp_scores():
    """Several key tiles per row, and scores of a spread of 16, so that the
    running maximum moves by more than its rescale threshold."""
    lens = [1000]
    x = make(14, "bf16", 2, 128, 64, lens, lens)
    check_all("1000 tokens", x, both(x, lens, lens, True), lens, lens, True)
    x["q"] = (x["q"].float() * 16).bfloat16()
    want = ref.attention(x["q"], x["k"], x["v"], x["k_pe"], lens, lens, True, x["scale"])
    got = both(x, lens, lens, True)
    ref.check("sharp o", got["o"], *want["o"])


def test_scores_far_from_zero():
    """All scores near +-300 (exp of them overflows or vanishes on its own)."""
    lens = [130]
    for sign in (1.0, -1.0):
        x = make(15, "f32", 2, 64, 0, lens, lens, spread=0.1)
        x["q"][..., 0] = 100.0
        x["k"][..., 0] = sign * 24.0
        # q . k is near 2400, where half a step of fp32 is 2^-13: the 64 additions
        # of the product are off by at most 64 * 2^-13 = 2^-7, a score (times
        # the scale 1/8) and with it a weight, relatively, by 2^-10, in any
        # fp32 evaluation, on top of the usual slack
        got = both(x, lens, lens, True)
        want = ref.attention(x["q"], x["k"], x["v"], None, lens, lens, True, x["scale"],
                             slack=ref.SLACK + 2.0 ** -10)
        ref.check(f"far {sign} o", got["o"], *want["o"])


def test_strided_inputs_and_given_outputs():
    """q inside a wider projection, k, v and their gradients halves of one
    tensor, k_pe a column range; heads-first storage."""
    import gated_delta_rule_prefill_amd as kda
    lens, H, d, dr = [100, 31], 4, 128, 64
    x = make(16, "bf16", H, d, dr, lens, lens)
    T = sum(lens)
    wide = torch.zeros(T, H, d + dr + 64, dtype=torch.bfloat16, device="cuda")
    wide[..., :d + dr] = x["q"]
    pe = torch.zeros(T, 640, dtype=torch.bfloat16, device="cuda")
    pe[:, 512:576] = x["k_pe"]
    hf = x["k"].transpose(0, 1).contiguous().transpose(0, 1)      # [T, H, d] stored heads first
    cu = offsets(lens)
    o0, l0 = kda.latent_attention(x["q"], x["k"], x["v"], k_pe=x["k_pe"], cu_seqlens=cu)
    o1, l1 = kda.latent_attention(wide[..., :d + dr], hf, x["v"], k_pe=pe[:, 512:576], cu_seqlens=cu)
    assert torch.equal(o0, o1) and torch.equal(l0, l1)
    g0 = kda.latent_attention_backward(x["q"], x["k"], x["v"], o0, l0, x["d_o"], k_pe=x["k_pe"], cu_seqlens=cu)
    dk, dv = (torch.full((H, T, d), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(0, 1) for _ in range(2))
    g1 = kda.latent_attention_backward(wide[..., :d + dr], hf, x["v"], o0, l0, x["d_o"], k_pe=pe[:, 512:576],
                                       cu_seqlens=cu, dk=dk, dv=dv)
    for n in g0:
        assert torch.equal(g0[n], g1[n]), n


def test_rows_behind_the_last_sequence_are_left():
    import gated_delta_rule_prefill_amd as kda
    lens = [70, 3]
    x = make(17, "bf16", 2, 128, 64, lens, lens, behind=77)
    n = sum(lens)
    for name in ("q", "k", "v", "k_pe", "d_o"):
        x[name][n:] = float("nan")
    cu = offsets(lens)
    out = torch.full((n + 77, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 77, 2), 7.0, device="cuda")
    kda.latent_attention(x["q"], x["k"], x["v"], k_pe=x["k_pe"], cu_seqlens=cu, out=out, lse=lse)
    dk, dv = (torch.full((n + 77, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = kda.latent_attention_backward(x["q"], x["k"], x["v"], out, lse, x["d_o"], k_pe=x["k_pe"], cu_seqlens=cu, dk=dk,
                                      dv=dv)
    for t in (out, lse, dk, dv):
        assert (t[n:] == 7.0).all()
    want = ref.attention(x["q"][:n], x["k"][:n], x["v"][:n], x["k_pe"][:n], lens, lens, True, x["scale"], x["d_o"][:n])
    for name, t in (("o", out), ("lse", lse), ("dk", dk), ("dv", dv), ("dq", g["dq"]), ("dk_pe", g["dk_pe"])):
        ref.check(f"padded {name}", t[:n], *want[name])


def test_many_short_sequences():
    """More sequences than a workgroup has threads."""
    lens = [(7 * i) % 5 for i in range(700)]
    x = make(18, "bf16", 8, 64, 64, lens, lens)
    check_all("700 sequences", x, both(x, lens, lens, True), lens, lens, True)


def test_gradients_against_differences():
    """fp32: a directional derivative of sum(o * d_o) by central differences of
    the forward kernel.  Step h = 2^-6 on unit directions: the kernel's fp32
    error of the sum, about 1e-6 sqrt(n), over 2h, and h^2 times the third
    derivative (a few units here), stay under 2 % of the derivative's scale."""
    import gated_delta_rule_prefill_amd as kda
    lens = [90, 40]
    x = make(19, "f32", 2, 64, 64, lens, lens, spread=0.5)
    cu = offsets(lens)
    got = both(x, lens, lens, True)
    f = lambda q, k, v, pe: float((kda.latent_attention(q, k, v, k_pe=pe, cu_seqlens=cu, scale=x["scale"])[0].double() *  # noqa: E731
                                   x["d_o"].double()).sum())
    names = {"q": "dq", "k": "dk", "v": "dv", "k_pe": "dk_pe"}
    gen = torch.Generator().manual_seed(5)
    for name, gname in names.items():
        direction = torch.randn(x[name].shape, generator=gen).cuda()
        direction /= direction.norm()
        # along the gradient's own direction too: its derivative is the gradient's norm
        for way in (direction, got[gname].float() / got[gname].float().norm()):
            h = 2.0 ** -6
            at = lambda s: f(*[x[n] + s * h * way if n == name else x[n] for n in names])  # noqa: E731
            diff = (at(1.0) - at(-1.0)) / (2 * h)
            dot = float((got[gname].double() * way.double()).sum())
            print(f"[latent] d/d{name}: {dot:.5f} by formula, {diff:.5f} by differences", flush=True)
            assert abs(diff - dot) <= 0.02 * float(got[gname].double().norm())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_replays_match_eager(dtype):
    """Forward and backward captured once and replayed on new inputs, eager
    calls in between; both deterministic, so bit for bit."""
    import gated_delta_rule_prefill_amd as kda
    lens = [130, 1, 64]
    cu = offsets(lens)
    xs = [make(20 + i, dtype, 4, 128, 64, lens, lens) for i in range(3)]
    s = {n: (t.clone() if isinstance(t, torch.Tensor) else t) for n, t in xs[0].items()}

    def step(x):
        o, lse = kda.latent_attention(x["q"], x["k"], x["v"], k_pe=x["k_pe"], cu_seqlens=cu)
        return [o, lse] + list(kda.latent_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], k_pe=x["k_pe"],
                                                             cu_seqlens=cu).values())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(s)
    for x in xs + xs:
        want = step(x)
        for n in ("q", "k", "v", "k_pe", "d_o"):
            s[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_other_stream():
    """The stream argument: the call and its allocations run there."""
    import gated_delta_rule_prefill_amd as kda
    lens = [300]
    x = make(24, "bf16", 4, 128, 64, lens, lens)
    want = both(x, lens, lens, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(x, lens, lens, True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for n in want:
        assert torch.equal(want[n], got[n]), n


def test_workspace_of_the_library():
    """NULL workspace through the C ABI: allocated on the stream; the same gradients."""
    from gated_delta_rule_prefill_amd import kda as b
    lens = [65, 20]
    x = make(25, "bf16", 2, 128, 64, lens, lens)
    want = both(x, lens, lens, True)
    cu = offsets(lens)
    a, _ = b._latent_inputs(x["q"], x["k"], x["v"], x["k_pe"], cu, None, None, True, x["scale"])
    got = {n: torch.empty_like(t).contiguous() for n, t in want.items()}
    dk, dv = got["dk"], got["dv"]
    st = b.lib().kda_latent_attention_backward(
        a, want["o"].data_ptr(), want["lse"].data_ptr(), x["d_o"].data_ptr(), got["dq"].data_ptr(),
        dk.data_ptr(), dk.stride(0), dk.stride(1), dv.data_ptr(), dv.stride(0), dv.stride(1), got["dk_pe"].data_ptr(),
        None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == b.KDA_OK, b.last_error()
    torch.cuda.synchronize()
    for n in ("dq", "dk", "dv", "dk_pe"):
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what,value", [("k", "nan"), ("v", "nan"), ("v", "inf"), ("k_pe", "inf"), ("k", "-inf")])
def test_hidden_keys_that_are_not_finite(dtype, what, value):
    """NaN or Inf in keys that the causal mask hides reaches no output or
    gradient of the rows before them; the rows that see them get NaN."""
    lens, bad = [200, 70], 150
    x = make(26, dtype, 2, 128, 64, lens, lens)
    clean = {n: (t.clone() if isinstance(t, torch.Tensor) else t) for n, t in x.items()}
    kv = torch.cat([x["k"], x["v"]], dim=2)
    x["k"], x["v"] = kv[..., :128], kv[..., 128:]
    x[what][bad, ..., 5] = float(value)
    x[what][199, ..., 63] = float(value)
    got = both(x, lens, lens, True)
    want = ref.attention(clean["q"], clean["k"], clean["v"], clean["k_pe"], lens, lens, True, x["scale"], x["d_o"])
    for name in ("o", "lse", "dq"):
        value_, bound = want[name]
        for part in (slice(0, bad), slice(200, 270)):
            ref.check(f"hidden {what} {value} {name}", got[name][part], value_[part], bound[part])
    if value == "nan":
        assert torch.isnan(got["o"][bad:200].float()).any(dim=-1).all()
        assert torch.isnan(got["dq"][bad:200].float()).any(dim=-1).all()
    # the other sequence's keys are untouched
    for name in ("dk", "dv", "dk_pe"):
        ref.check(f"other sequence {name}", got[name][200:], want[name][0][200:], want[name][1][200:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["q", "d_o"])
def test_rows_that_are_not_finite_leave_later_keys_clean(dtype, what):
    """A query row with NaN spoils the gradients of the keys it sees, not of the
    keys behind it."""
    lens, bad = [200], 20
    x = make(27, dtype, 2, 128, 64, lens, lens)
    clean = {n: (t.clone() if isinstance(t, torch.Tensor) else t) for n, t in x.items()}
    clean["q"][bad] = 0.0
    clean["d_o"][bad] = 0.0      # the row adds nothing
    x[what][bad, 0, 3] = float("nan")
    x[what][bad, 1, 100] = float("inf")
    got = both(x, lens, lens, True)
    want = ref.attention(clean["q"], clean["k"], clean["v"], clean["k_pe"], lens, lens, True, x["scale"], clean["d_o"])
    for name in ("dk", "dv", "dk_pe"):
        ref.check(f"keys behind a bad {what} {name}", got[name][bad + 1:], want[name][0][bad + 1:], want[name][1][bad + 1:])
    rows = torch.arange(200) != bad
    for name in ("o", "dq") if what == "q" else ("dq",):
        ref.check(f"other rows {name}", got[name][rows.cuda()], want[name][0][rows], want[name][1][rows])


def test_padded_rows_of_garbage():
    """Equal rows padded on the right with NaN: the rows before the padding."""
    import gated_delta_rule_prefill_amd as kda
    lens, n = [128, 128, 128], [100, 1, 127]
    x = make(28, "bf16", 4, 128, 64, lens, lens)
    want = ref.attention(x["q"], x["k"], x["v"], x["k_pe"], lens, lens, True, x["scale"])
    for i, m in enumerate(n):
        for name in ("q", "k", "v", "k_pe"):
            x[name][128 * i + m:128 * (i + 1)] = float("nan")
    o, lse = kda.latent_attention(x["q"], x["k"], x["v"], k_pe=x["k_pe"], num_seqs=3, scale=x["scale"])
    for i, m in enumerate(n):
        part = slice(128 * i, 128 * i + m)
        ref.check(f"padded row {i} o", o[part], want["o"][0][part], want["o"][1][part])
        ref.check(f"padded row {i} lse", lse[part], want["lse"][0][part], want["lse"][1][part])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens_q,lens_k", [([70, 40], [20, 33]), ([150, 9], [140, 0])])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_rows_without_keys_and_gradients_that_are_not_finite(dtype, lens_q, lens_k, value):
    """Rows that see no key have zero gradients whatever d_o holds there, in the
    same wave as rows that see keys or not, and leave the keys' gradients clean."""
    x = make(29, dtype, 2, 128, 64, lens_q, lens_k)
    clean = dict(x, d_o=x["d_o"].clone())
    at, empty = 0, []
    for n, m in zip(lens_q, lens_k):
        empty += range(at, at + n - m)
        at += n
    x["d_o"][empty, :, 5] = float(value)
    x["d_o"][empty[::2]] = float(value)
    clean["d_o"][empty] = 0.0
    got = both(x, lens_q, lens_k, True)
    check_all(f"no keys, d_o {value} {dtype}", clean, got, lens_q, lens_k, True)
    assert (got["dq"][empty] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,dr", [(128, 64), (64, 0)])
@pytest.mark.parametrize("causal", [True, False])
def test_values_of_infinity_reach_their_channel_only(dtype, d, dr, causal):
    """Inf and NaN in a value reach that channel of the rows that see it, in
    every tile alike; the other channels and lse are those without it."""
    import gated_delta_rule_prefill_amd as kda
    lens, first = [400, 70], [0, 400]
    x = make(30, dtype, 3, d, dr, lens, lens)
    bad = [(0, 3, 1, 9, math.inf), (0, 150, 0, 5, -math.inf), (0, 151, 2, 7, math.nan), (0, 399, 1, 60, math.inf),
           (1, 64, 0, 0, math.nan)]
    v = x["v"].clone()
    for s, j, h, c, value in bad:
        x["v"][first[s] + j, h, c] = value
        v[first[s] + j, h, c] = 0.0
    o, lse = kda.latent_attention(x["q"], x["k"], x["v"], k_pe=x["k_pe"], cu_seqlens=offsets(lens), causal=causal,
                                  scale=x["scale"])
    want = ref.attention(x["q"], x["k"], v, x["k_pe"], lens, lens, causal, x["scale"])
    ref.check("lse", lse, *want["lse"])
    o = o.double().cpu()
    for s, j, h, c, value in bad:
        rows = slice(first[s] + (j if causal else 0), first[s] + lens[s])
        seen = o[rows, h, c]
        assert torch.equal(torch.nan_to_num(seen, 1.0, 2.0, 3.0),
                           torch.nan_to_num(torch.full_like(seen, value), 1.0, 2.0, 3.0)), (s, j, h, c)
        o[rows, h, c] = want["o"][0][rows, h, c]
    ref.check("o elsewhere", o, *want["o"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,dr", [(128, 64), (128, 0), (64, 64), (64, 0)])
@pytest.mark.parametrize("lens_q,lens_k", [([70, 300, 1], [500, 200, 129]), ([257, 33], [257, 33]), ([300, 64], [40, 64])])
@pytest.mark.parametrize("causal", [True, False])
def test_values_that_are_not_finite_anywhere(dtype, d, dr, lens_q, lens_k, causal):
    """Inf, -Inf and NaN strewn over the values: each channel of a row is what
    the values it sees make of it, whatever tiles they lie in."""
    import gated_delta_rule_prefill_amd as kda
    H = 3
    x = make(32, dtype, H, d, dr, lens_q, lens_k)
    g = torch.Generator().manual_seed(33)
    odd = torch.randint(0, 400, x["v"].shape, generator=g).cuda()      # 0.75 % of the values
    clean = x["v"].masked_fill(odd < 3, 0.0)
    for i, value in enumerate((math.inf, -math.inf, math.nan)):
        x["v"].masked_fill_(odd == i, value)
    o, lse = kda.latent_attention(x["q"], x["k"], x["v"], k_pe=x["k_pe"], cu_seqlens=offsets(lens_q),
                                  cu_seqlens_k=offsets(lens_k), causal=causal, scale=x["scale"])
    want = ref.attention(x["q"], x["k"], clean, x["k_pe"], lens_q, lens_k, causal, x["scale"])
    ref.check("lse", lse, *want["lse"])
    value, bound = want["o"]
    a = b = 0
    for n, m in zip(lens_q, lens_k):
        i, j = torch.arange(n)[:, None], torch.arange(m)[None]
        sees = ((j <= i + (m - n)) if causal else (j >= 0)).expand(n, m).double()
        up, down = (torch.einsum("nm,mhc->nhc", sees, ((odd[b:b + m] == s) | (odd[b:b + m] == 2)).double().cpu()) > 0
                    for s in (0, 1))
        part = value[a:a + n]
        part[up], part[down], part[up & down] = math.inf, -math.inf, math.nan
        a, b = a + n, b + m
    got = o.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(value))
    there = ~torch.isnan(value)
    ref.check("o", got.masked_fill(~there, 0.0), value.masked_fill(~there, 0.0), bound)
