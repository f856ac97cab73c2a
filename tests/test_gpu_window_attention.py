"""Window attention and its gradients against the definition in float64, element
by element (bounds in window_reference.py)."""
import math

import pytest
import torch

import window_reference as ref
from test_gpu_guards import Guarded, _check

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def offsets(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def make(seed, dtype, H, Hk, d, lens_q, lens_k, behind=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    T, Tk = sum(lens_q) + behind, sum(lens_k) + behind
    r = lambda *s: (torch.randn(*s, generator=g) * spread).to(DT[dtype]).cuda()  # noqa: E731
    kv = r(Tk, 2 * Hk, d)
    return dict(q=r(T, H, d), k=kv[:, :Hk], v=kv[:, Hk:], d_o=r(T, H, d))


def both(x, lens_q, lens_k, window, sinks, packed=True, **kw):
    import gated_delta_rule_prefill_amd as kda
    args = dict(window=window, sinks=sinks, **kw)
    if packed:
        args["cu_seqlens"] = offsets(lens_q)
        if lens_k != lens_q:
            args["cu_seqlens_k"] = offsets(lens_k)
    else:
        args["num_seqs"] = len(lens_q)
    o, lse = kda.window_attention(x["q"], x["k"], x["v"], **args)
    grads = kda.window_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], **args)
    torch.cuda.synchronize()
    return dict(o=o, lse=lse, **grads)


def check_all(label, x, got, lens_q, lens_k, window, sinks):
    want = ref.attention(x["q"], x["k"], x["v"], lens_q, lens_k, window, sinks, d_o=x["d_o"])
    T, Tk = sum(lens_q), sum(lens_k)
    for name, (value, bound) in want.items():
        n = T if name in ("o", "lse", "dq") else Tk
        ref.check(f"{label} {name}", got[name][:n], value[:n], bound[:n])


RAGGED = [1, 0, 63, 64, 65, 128, 129, 2, 200]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,d", [(3, 3, 128), (8, 2, 64), (5, 1, 128), (12, 3, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 4), (64, 0), (100, 64), (2 ** 31 - 1, 3)])
def test_ragged_batch(dtype, H, Hk, d, window, sinks):
    x = make(11, dtype, H, Hk, d, RAGGED, RAGGED)
    check_all(f"ragged {dtype} {H}/{Hk} {d} W={window} S={sinks}", x, both(x, RAGGED, RAGGED, window, sinks), RAGGED,
              RAGGED, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens_q,lens_k", [
    ([5, 1, 70, 0, 33], [40, 130, 70, 9, 300]),      # new tokens after a kept prefix; keys without queries
    ([70, 130, 3], [20, 129, 0]),                    # rows that see no key
])
@pytest.mark.parametrize("window,sinks", [(1, 0), (32, 2), (150, 64)])
def test_unequal_lengths(dtype, lens_q, lens_k, window, sinks):
    x = make(12, dtype, 8, 2, 128, lens_q, lens_k)
    check_all(f"unequal {dtype} {lens_q} {lens_k} W={window}", x, both(x, lens_q, lens_k, window, sinks), lens_q,
              lens_k, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_rows_and_one_token(dtype):
    for lens in ([1], [97, 97, 97], [256, 256]):
        x = make(13, dtype, 4, 2, 64, lens, lens)
        check_all(f"rows {dtype} {lens}", x, both(x, lens, lens, 50, 4, packed=False), lens, lens, 50, 4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sinks", [1, 17, 64])
def test_sinks_of_long_sequences(dtype, sinks):
    """The sinks' gradients come in pieces of 1,024 tokens: none, one and three of
    them, the last one short, in one batch."""
    lens, window = [150, 1300, 2390], 100
    x = make(14, dtype, 2, 1, 64, lens, lens)
    check_all(f"long {dtype} S={sinks}", x, both(x, lens, lens, window, sinks), lens, lens, window, sinks)


def test_pieces_behind_a_prefix():
    """Queries that all stand behind the first tile's window, and some that do not."""
    lens_q, lens_k = [1100, 40, 1025], [3000, 90, 1200]
    x = make(15, "bf16", 4, 2, 128, lens_q, lens_k)
    check_all("prefix", x, both(x, lens_q, lens_k, 64, 4), lens_q, lens_k, 64, 4)


@pytest.mark.parametrize("H,Hk", [(8, 8), (16, 8), (14, 2), (9, 9)])
def test_head_counts(H, Hk):
    lens = [257, 1, 90]
    x = make(16, "bf16", H, Hk, 128, lens, lens)
    check_all(f"{H}/{Hk}", x, both(x, lens, lens, 70, 5), lens, lens, 70, 5)


def test_sharp_scores():
    """Scores of a spread of 16: the running maximum moves by more than its rescale threshold."""
    lens = [700]
    x = make(17, "bf16", 2, 2, 128, lens, lens)
    x["q"] = (x["q"].float() * 16).bfloat16()
    want = ref.attention(x["q"], x["k"], x["v"], lens, lens, 300, 4)
    ref.check("sharp o", both(x, lens, lens, 300, 4)["o"], *want["o"])


def test_strided_inputs_and_given_outputs():
    """Parts of one projection, heads-first storage, gradients into a wider tensor."""
    import gated_delta_rule_prefill_amd as kda
    lens, H, Hk, d = [100, 31], 4, 2, 128
    x = make(18, "bf16", H, Hk, d, lens, lens)
    T, cu = sum(lens), offsets(lens)
    args = dict(window=40, sinks=3, cu_seqlens=cu)
    wide = torch.zeros(T, H + 2 * Hk, d, dtype=torch.bfloat16, device="cuda")
    wide[:, :H], wide[:, H:H + Hk] = x["q"], x["k"]
    hf = x["v"].transpose(0, 1).contiguous().transpose(0, 1)
    o0, l0 = kda.window_attention(x["q"], x["k"], x["v"], **args)
    o1, l1 = kda.window_attention(wide[:, :H], wide[:, H:H + Hk], hf, **args)
    assert torch.equal(o0, o1) and torch.equal(l0, l1)
    g0 = kda.window_attention_backward(x["q"], x["k"], x["v"], o0, l0, x["d_o"], **args)
    grad = torch.full((T, H + 2 * Hk, d), 7.0, dtype=torch.bfloat16, device="cuda")
    g1 = kda.window_attention_backward(wide[:, :H], wide[:, H:H + Hk], hf, o0, l0, x["d_o"], dk=grad[:, H:H + Hk],
                                       dv=grad[:, H + Hk:], **args)
    for n in g0:
        assert torch.equal(g0[n], g1[n]), n
    assert (grad[:, :H] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sinks", [0, 9])
def test_writes_stay_in_bounds(dtype, sinks):
    import gated_delta_rule_prefill_amd as kda
    lens, H, Hk, d, t = [1, 65, 0, 1330], 3, 3, 64, DT[dtype]
    x = make(19, dtype, H, Hk, d, lens, lens)
    T = sum(lens)
    args = dict(window=33, sinks=sinks, cu_seqlens=offsets(lens))
    out = dict(o=Guarded((T, H, d), t), lse=Guarded((T, H), torch.float32))
    o, lse = kda.window_attention(x["q"], x["k"], x["v"], out=out["o"].t, lse=out["lse"].t, **args)
    need = kda.window_attention_backward_workspace_bytes(T, 4, H, Hk, d, sinks)
    out.update(dk=Guarded((T, Hk, d), t), dv=Guarded((T, Hk, d), t),
               ws=Guarded((need,), torch.uint8, init=torch.full((need,), 255, dtype=torch.uint8, device="cuda")))
    grads = kda.window_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], dk=out["dk"].t, dv=out["dv"].t,
                                          workspace=out["ws"].t, **args)
    _check(out, f"window attention {dtype}")
    check_all("guarded", x, dict(o=o, lse=lse, **grads), lens, lens, 33, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_outside_the_sequences_are_left(dtype):
    """Offsets that start late and end early: the rows before and behind are neither read nor written."""
    import gated_delta_rule_prefill_amd as kda
    lens, first, behind, H, Hk, d = [70, 130], 5, 7, 4, 2, 64
    x = make(20, dtype, H, Hk, d, lens, lens, behind=first + behind)
    n = sum(lens)
    for name in ("q", "k", "v", "d_o"):
        x[name][:first] = float("nan")
        x[name][first + n:] = float("nan")
    cu = offsets(lens) + first
    T = first + n + behind
    mark = lambda *s: torch.full(s, 7.0, dtype=DT[dtype], device="cuda")  # noqa: E731
    o, dk, dv, lse = mark(T, H, d), mark(T, Hk, d), mark(T, Hk, d), torch.full((T, H), 7.0, device="cuda")
    args = dict(window=50, sinks=2, cu_seqlens=cu)
    kda.window_attention(x["q"], x["k"], x["v"], out=o, lse=lse, **args)
    g = kda.window_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], dk=dk, dv=dv, **args)
    part = slice(first, first + n)
    check_all("inside", {m: t[part] for m, t in x.items()}, {m: t[part] for m, t in dict(o=o, lse=lse, **g).items()},
              lens, lens, 50, 2)
    for t in (o, lse, dk, dv):
        assert (t[:first] == 7.0).all() and (t[first + n:] == 7.0).all()


def test_many_short_sequences():
    lens = [(7 * i) % 5 for i in range(700)]
    x = make(21, "bf16", 8, 4, 64, lens, lens)
    check_all("700 sequences", x, both(x, lens, lens, 2, 1), lens, lens, 2, 1)


def test_nothing_to_do():
    """No tokens, sequences without tokens, keys without queries."""
    import gated_delta_rule_prefill_amd as kda
    x = make(22, "bf16", 4, 2, 64, [0], [0])
    got = both(x, [0, 0], [0, 0], 5, 2)
    assert got["o"].shape == (0, 4, 64) and got["dk"].shape == (0, 2, 64)
    x = make(22, "bf16", 4, 2, 64, [0], [90])
    got = both(x, [0, 0], [60, 30], 5, 2)
    assert (got["dk"] == 0).all() and (got["dv"] == 0).all()
    x = make(22, "bf16", 4, 2, 64, [90], [0])
    got = both(x, [60, 30], [0, 0], 5, 2)
    assert (got["o"] == 0).all() and torch.isneginf(got["lse"]).all() and (got["dq"] == 0).all()
    assert kda.window_attention(x["q"][:0], x["q"][:0, :2], x["q"][:0, :2], window=1)[0].shape == (0, 4, 64)


def test_gradients_against_differences():
    """fp32: a directional derivative of sum(o * d_o) by central differences of
    the forward kernel.  Step h = 2^-6 on unit directions: the kernel's fp32
    error of the sum, about 1e-6 sqrt(n), over 2h, and h^2 times the third
    derivative (a few units here), stay under 2 % of the derivative's scale."""
    import gated_delta_rule_prefill_amd as kda
    lens = [90, 240]
    x = make(23, "f32", 4, 2, 64, lens, lens, spread=0.5)
    args = dict(window=40, sinks=4, cu_seqlens=offsets(lens))
    got = both(x, lens, lens, 40, 4)
    f = lambda q, k, v: float((kda.window_attention(q, k, v, **args)[0].double() * x["d_o"].double()).sum())  # noqa: E731
    gen = torch.Generator().manual_seed(5)
    for name, gname in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        direction = torch.randn(x[name].shape, generator=gen).cuda()
        direction /= direction.norm()
        # along the gradient's own direction too: its derivative is the gradient's norm
        for way in (direction, got[gname].float() / got[gname].float().norm()):
            h = 2.0 ** -6
            at = lambda s: f(*[x[n] + s * h * way if n == name else x[n] for n in ("q", "k", "v")])  # noqa: E731
            diff = (at(1.0) - at(-1.0)) / (2 * h)
            dot = float((got[gname].double() * way.double()).sum())
            print(f"[window] d/d{name}: {dot:.5f} by formula, {diff:.5f} by differences", flush=True)
            assert abs(diff - dot) <= 0.02 * float(got[gname].double().norm())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_replays_match_eager(dtype):
    """Forward and backward captured once and replayed on new inputs, eager calls
    in between; both deterministic, so bit for bit."""
    import gated_delta_rule_prefill_amd as kda
    lens = [1300, 1, 64]
    args = dict(window=70, sinks=4, cu_seqlens=offsets(lens))
    xs = [make(24 + i, dtype, 4, 2, 128, lens, lens) for i in range(3)]
    s = {n: t.clone() for n, t in xs[0].items()}

    def step(x):
        o, lse = kda.window_attention(x["q"], x["k"], x["v"], **args)
        return [o, lse] + list(kda.window_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], **args).values())
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
        for n in s:
            s[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_other_stream_and_calls_at_the_same_time():
    """Training steps on two streams at once, each on its own inputs, give what they give alone."""
    lens = [1500, 300]
    xs = [make(27 + i, "bf16", 8, 2, 128, lens, lens) for i in range(2)]
    want = [both(x, lens, lens, 200, 4) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    import gated_delta_rule_prefill_amd as kda
    cu, got = offsets(lens), []
    torch.cuda.synchronize()
    for x, stream in zip(xs, (None, side)):
        args = dict(window=200, sinks=4, cu_seqlens=cu, stream=stream)
        o, lse = kda.window_attention(x["q"], x["k"], x["v"], **args)
        got.append(dict(o=o, lse=lse, **kda.window_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], **args)))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for n in a:
            assert torch.equal(a[n], b[n]), n


def test_workspace_of_the_library():
    """NULL workspace through the C ABI: allocated on the stream; the same gradients."""
    from gated_delta_rule_prefill_amd import kda as b
    lens = [65, 1300]
    x = make(29, "bf16", 2, 2, 128, lens, lens)
    want = both(x, lens, lens, 60, 4)
    a, _ = b._window_inputs(x["q"], x["k"], x["v"], 60, 4, offsets(lens), None, None, None)
    dq, dk, dv = (torch.empty(x["q"].shape, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    cu = offsets(lens)
    a, _ = b._window_inputs(x["q"], x["k"], x["v"], 60, 4, cu, None, None, None)
    st = b.lib().kda_window_attention_backward(
        a, want["o"].data_ptr(), want["lse"].data_ptr(), x["d_o"].data_ptr(), dq.data_ptr(), dk.data_ptr(), dk.stride(0),
        dk.stride(1), dv.data_ptr(), dv.stride(0), dv.stride(1), None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == b.KDA_OK, b.last_error()
    torch.cuda.synchronize()
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(t, want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what,value", [("k", "nan"), ("v", "nan"), ("v", "inf"), ("k", "-inf")])
@pytest.mark.parametrize("window,sinks", [(40, 4), (40, 64)])
def test_hidden_keys_that_are_not_finite(dtype, what, value, window, sinks):
    """NaN or Inf in a key reaches no output or gradient of the rows that do not
    see it, before it or beyond its window; the rows that see it get NaN."""
    lens, bad = [200, 70], 100
    x = make(30, dtype, 4, 2, 128, lens, lens)
    clean = {n: t.clone() for n, t in x.items()}
    x[what][bad, :, 5] = float(value)
    got = both(x, lens, lens, window, sinks)
    want = ref.attention(clean["q"], clean["k"], clean["v"], lens, lens, window, sinks, d_o=clean["d_o"])
    for name in ("o", "lse", "dq"):
        for part in (slice(0, bad), slice(bad + window, 270)):
            ref.check(f"hidden {what} {value} {name}", got[name][part], want[name][0][part], want[name][1][part])
    if value == "nan":
        assert torch.isnan(got["o"][bad:bad + window].float()).any(dim=-1).all()
        assert torch.isnan(got["dq"][bad:bad + window].float()).any(dim=-1).all()
    for name in ("dk", "dv"):   # the other sequence, and keys that no row sees which sees the bad one
        for part in (slice(200, 270), slice(sinks, bad - window), slice(bad + window, 200)):
            ref.check(f"other keys {name}", got[name][part], want[name][0][part], want[name][1][part])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["q", "d_o"])
def test_rows_that_are_not_finite_leave_hidden_keys_clean(dtype, what):
    """A query row with NaN spoils the gradients of the keys it sees only."""
    lens, bad, window, sinks = [300], 150, 60, 4
    x = make(31, dtype, 4, 2, 128, lens, lens)
    clean = {n: t.clone() for n, t in x.items()}
    clean["q"][bad] = 0.0
    clean["d_o"][bad] = 0.0      # the row adds nothing
    x[what][bad, 0, 3] = float("nan")
    x[what][bad, 2:, 100] = float("inf")
    got = both(x, lens, lens, window, sinks)
    want = ref.attention(clean["q"], clean["k"], clean["v"], lens, lens, window, sinks, d_o=clean["d_o"])
    for name in ("dk", "dv"):
        for part in (slice(bad + 1, 300), slice(sinks, bad - window + 1)):
            ref.check(f"keys hidden from a bad {what} {name}", got[name][part], want[name][0][part], want[name][1][part])
    rows = torch.arange(300) != bad
    for name in ("o", "dq") if what == "q" else ("dq",):
        ref.check(f"other rows {name}", got[name][rows.cuda()], want[name][0][rows], want[name][1][rows])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_rows_without_keys_and_gradients_that_are_not_finite(dtype, value):
    """Rows that see no key have zero gradients whatever d_o holds there."""
    lens_q, lens_k = [150, 70], [100, 33]
    x = make(32, dtype, 4, 2, 128, lens_q, lens_k)
    clean = dict(x, d_o=x["d_o"].clone())
    empty = list(range(50)) + list(range(150, 187))
    x["d_o"][empty, :, 5] = float(value)
    clean["d_o"][empty] = 0.0
    got = both(x, lens_q, lens_k, 30, 2)
    check_all(f"no keys, d_o {value}", clean, got, lens_q, lens_k, 30, 2)
    assert (got["dq"][empty] == 0).all()


def test_offsets_beyond_32_bits():
    """Keys and queries far apart in one large buffer: element offsets beyond 2^31."""
    import gated_delta_rule_prefill_amd as kda
    H, Hk, d, T = 4, 2, 64, 300
    x = make(33, "bf16", H, Hk, d, [T], [T])
    stride = (1 << 23) - 64
    big = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    far = lambda t, at: torch.as_strided(big, t.shape, (stride, d, 1), at).copy_(t)  # noqa: E731
    q, k, v = far(x["q"], 0), far(x["k"], 1024), far(x["v"], 2048)
    args = dict(window=100, sinks=4)
    o, lse = kda.window_attention(q, k, v, **args)
    g = kda.window_attention_backward(q, k, v, o, lse, x["d_o"], dk=torch.as_strided(big, (T, Hk, d), (stride, d, 1), 4096),
                                      dv=torch.as_strided(big, (T, Hk, d), (stride, d, 1), 8192), **args)
    check_all("far", x, dict(o=o, lse=lse, **g), [T], [T], 100, 4)
    assert math.isfinite(float(o.float().sum()))
