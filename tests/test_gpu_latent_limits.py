"""Latent attention at its limits: guard bytes around every output, workspaces
that hold anything, offsets that do not start at 0, head counts that no tile
divides, and calls that run at the same time."""
import pytest
import torch

import latent_reference as ref
import test_gpu_latent_attention as ta
import test_gpu_latent_decode as td
from test_gpu_guards import PATTERN, Guarded, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ones(n):
    """A workspace whose every word is NaN, as bf16 and as fp32."""
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dr", [64, 0])
def test_attention_writes_stay_in_bounds(dtype, dr):
    import gated_delta_rule_prefill_amd as kda
    from gated_delta_rule_prefill_amd import kda as b
    lens, H, d = [1, 65, 0, 130], 3, 64
    x = ta.make(60, dtype, H, d, dr, lens, lens)
    T, t = sum(lens), ta.DT[dtype]
    args = dict(k_pe=x["k_pe"], cu_seqlens=ta.offsets(lens), scale=x["scale"])
    out = dict(o=Guarded((T, H, d), t), lse=Guarded((T, H), torch.float32))
    o, lse = kda.latent_attention(x["q"], x["k"], x["v"], out=out["o"].t, lse=out["lse"].t, **args)
    need = b.lib().kda_latent_attention_backward_workspace_bytes(T, T, H, dr)
    out.update(dk=Guarded((T, H, d), t), dv=Guarded((T, H, d), t), ws=Guarded((need,), torch.uint8, init=ones(need)))
    grads = kda.latent_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], dk=out["dk"].t, dv=out["dv"].t,
                                          workspace=out["ws"].t, **args)
    _check(out, f"latent attention {dtype} dr={dr}")
    ta.check_all("guarded", x, dict(o=o, lse=lse, **grads), lens, lens, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,new", [(3, [1, 1, 1]), (32, [70, 0, 3])])
def test_decode_writes_stay_in_bounds(dtype, H, new):
    from gated_delta_rule_prefill_amd import kda as b
    lens = [300, 17, 64]
    x = td.make(61, dtype, H, 256, 64, 16, lens, new)
    T, t = sum(new), td.DT[dtype]
    need = b.latent_decode_workspace_bytes(T, 3, H, 256, 64, dtype == "bf16")
    out = dict(o=Guarded((T, H, 256), t), lse=Guarded((T, H), torch.float32),
               ws=Guarded((need,), torch.uint8, init=ones(need)))
    td.check("guarded", x, 256, lens, new, out=out["o"].t, lse=out["lse"].t, workspace=out["ws"].t)
    _check(out, f"latent decode {dtype} H={H}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_and_rotary_writes_stay_in_bounds(dtype):
    import gated_delta_rule_prefill_amd as kda
    t, dl, dr, page, lens, new = td.DT[dtype], 256, 64, 16, [20, 5], [7, 5]
    T = sum(new)
    g = torch.Generator().manual_seed(62)
    r = lambda *s: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    table = torch.tensor([[2, 0], [1, -1]], dtype=torch.int32, device="cuda")
    freq, _ = kda.rotary_frequencies(dr, device="cuda")
    out = dict(cache=Guarded((3, page, dl + dr), t), c=Guarded((T, dl), t), pe=Guarded((T, dr), t),
               y=Guarded((T, 3, 200), t))
    kda.latent_append(out["cache"].t, r(T, dl), table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      k_pe=r(T, dr), cu_seqlens=td.offsets(new), norm_weight=torch.ones(dl, device="cuda"),
                      inv_freq=freq, c_out=out["c"].t, k_pe_out=out["pe"].t)
    kda.rotary(r(T, 3, 200), torch.arange(T, dtype=torch.int32, device="cuda"), freq, start=104, out=out["y"].t)
    _check(out, f"latent append {dtype}")
    # of the cache only the new tokens' rows
    written = (out["cache"].t.view(torch.uint8) != PATTERN).reshape(3 * page, -1).any(dim=1).nonzero().flatten().tolist()
    rows = [16 * (2 if p < 16 else 0) + p % 16 for p in range(13, 20)] + [16 + p for p in range(5)]
    assert written == sorted(rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_that_start_late(dtype):
    """The first sequence starts behind row 0: the rows before it stay as they are."""
    import gated_delta_rule_prefill_amd as kda
    lens, first, H = [70, 130], 5, 5
    x = ta.make(63, dtype, H, 128, 64, lens, lens, behind=first)
    cu = ta.offsets(lens) + first
    mark = lambda *s: torch.full(s, 7.0, dtype=ta.DT[dtype], device="cuda")  # noqa: E731
    o, dk, dv = mark(205, H, 128), mark(205, H, 128), mark(205, H, 128)
    args = dict(k_pe=x["k_pe"], cu_seqlens=cu, scale=x["scale"])
    lse = torch.full((205, H), 7.0, device="cuda")
    kda.latent_attention(x["q"], x["k"], x["v"], out=o, lse=lse, **args)
    grads = kda.latent_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], dk=dk, dv=dv, **args)
    part = {n: t[first:] if t is not None and n != "scale" else t for n, t in x.items() if n != "scale"}
    part["scale"] = x["scale"]
    got = dict(o=o, lse=lse, **grads)
    ta.check_all("late", part, {n: t[first:] for n, t in got.items()}, lens, lens, True)
    for t in (o, lse, dk, dv):
        assert (t[:first] == 7.0).all()


@pytest.mark.parametrize("H", [3, 13, 16])
def test_head_counts(H):
    lens = [257, 1, 90]
    x = ta.make(64, "bf16", H, 128, 64, lens, lens)
    ta.check_all(f"H={H}", x, ta.both(x, lens, lens, True), lens, lens, True)


def test_more_new_tokens_than_cached_ones():
    """New tokens beyond the cache's length: the first of them see no key."""
    lens, new = [3, 0], [6, 2]
    x = td.make(65, "bf16", 2, 256, 64, 16, lens, new)
    td.check("more new than cached", x, 256, lens, new)
    o, lse = td.run(x, 256)
    assert (o[:3] == 0).all() and torch.isneginf(lse[:3]).all() and (o[6:] == 0).all()


def test_calls_at_the_same_time():
    """Decode and training steps on two streams at once, each with its own
    workspace, give what they give alone."""
    import gated_delta_rule_prefill_amd as kda
    lens, new = [5000, 700, 64], [1, 1, 1]
    xs = [td.make(66 + i, "bf16", 32, 512, 64, 64, lens, new) for i in range(2)]
    ts = [ta.make(68 + i, "bf16", 8, 128, 64, [300, 212], [300, 212]) for i in range(2)]

    def train(x):
        args = dict(k_pe=x["k_pe"], cu_seqlens=ta.offsets([300, 212]), scale=x["scale"])
        o, lse = kda.latent_attention(x["q"], x["k"], x["v"], **args)
        return kda.latent_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], **args)

    want = [(td.run(x, 512), train(y)) for x, y in zip(xs, ts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, x, y in zip(streams, xs, ts):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append((td.run(x, 512), train(y)))
        torch.cuda.synchronize()
        for (a, ga), (b, gb) in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            for n in ("dq", "dk", "dv", "dk_pe"):
                assert torch.equal(ga[n], gb[n])


def test_dirty_workspaces_change_nothing():
    """The library's own workspaces come from memory that held NaN."""
    from gated_delta_rule_prefill_amd import kda as b
    lens, new = [900, 64, 5, 1], [1, 1, 1, 1]
    x = td.make(70, "bf16", 32, 512, 64, 64, lens, new)
    need = b.latent_decode_workspace_bytes(4, 4, 32, 512, 64, True)
    got = td.run(x, 512, workspace=ones(need))
    want = td.run(x, 512, workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ref.check("dirty", got[0], *ref.decode(x["q"], x["cache"], x["table"], lens, new, 512, x["scale"])[0])


def test_grids_of_more_than_one_row():
    """Batches whose workgroups go into several rows of the grid end like the
    same tokens alone."""
    import gated_delta_rule_prefill_amd as kda
    g = torch.Generator(device="cuda").manual_seed(71)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    freq, _ = kda.rotary_frequencies(64, device="cuda")
    # rotary: a token a workgroup
    T, tail = 66000, 500
    x, pos = r(T, 32, 192), torch.arange(T, dtype=torch.int32, device="cuda")
    y = kda.rotary(x, pos, freq, start=128)
    assert torch.equal(y[-tail:], kda.rotary(x[-tail:].contiguous(), pos[-tail:].contiguous(), freq, start=128))
    # append: four tokens a workgroup, into one long sequence's pages
    T = 263000
    c, pe = r(T, 64), r(T, 64)
    table = torch.arange(-(-T // 64), dtype=torch.int32, device="cuda")[None]
    cache = torch.zeros(table.numel(), 64, 128, dtype=torch.bfloat16, device="cuda")
    kda.latent_append(cache, c, table, torch.tensor([T], dtype=torch.int32, device="cuda"), k_pe=pe, num_seqs=1)
    assert torch.equal(cache.view(-1, 128)[:T], torch.cat([c, pe], dim=1))
    # the sum of dk_pe: 16 keys a workgroup
    N, tail = 16500, 20
    T = 64 * N
    q, k, v, pe, do = r(T, 1, 128), r(T, 1, 64), r(T, 1, 64), r(T, 64), r(T, 1, 64)

    def step(a, n):
        part = [t[a:].contiguous() for t in (q, k, v, pe, do)]
        o, lse = kda.latent_attention(*part[:3], k_pe=part[3], num_seqs=n)
        return kda.latent_attention_backward(*part[:3], o, lse, part[4], k_pe=part[3], num_seqs=n)
    whole, alone = step(0, N), step(64 * (N - tail), tail)
    for n in ("dq", "dk", "dv", "dk_pe"):
        assert torch.equal(whole[n][-64 * tail:], alone[n])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_rotary_of_more_than_the_caches_hold(interleaved, in_place):
    """Outputs beyond 256 MB are stored another way: the same values."""
    import gated_delta_rule_prefill_amd as kda
    T, H, d = 33000, 32, 192 if not in_place else 128
    x = torch.randn(T, H, d, generator=torch.Generator(device="cuda").manual_seed(72), device="cuda").bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freq, _ = kda.rotary_frequencies(128, device="cuda")
    parts = [slice(0, 100), slice(16000, 16100), slice(T - 100, T)]
    want = [kda.rotary(x[p].contiguous(), pos[p].contiguous(), freq, start=d - 128, interleaved=interleaved) for p in parts]
    y = kda.rotary(x, pos, freq, start=d - 128, interleaved=interleaved, out=x if in_place else None)
    for p, w in zip(parts, want):
        assert torch.equal(y[p], w)


@pytest.mark.parametrize("lens_q,lens_k,H", [([2100], [2100], 4), ([700, 5, 0], [700, 5, 0], 3), ([64, 0], [9000, 70], 1),
                                             ([9000], [40], 1), ([1], [1], 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_fp32_gradients_split_and_whole(lens_q, lens_k, H, causal):
    """fp32 batches on either side of the size from which a tile's walk is no
    longer shared by several workgroups, queries and keys apart."""
    x = ta.make(73, "f32", H, 64, 64, lens_q, lens_k)
    ta.check_all("split", x, ta.both(x, lens_q, lens_k, causal), lens_q, lens_k, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_workspace_for_batches_of_any_size(dtype):
    """A workspace sized for the largest batch, reused for smaller ones, whose
    walks are split or whose row tiles are of another shape."""
    from gated_delta_rule_prefill_amd import kda as b
    need = b.lib().kda_latent_attention_backward_workspace_bytes(3000, 3000, 4, 64)
    ws = ones(need)
    import gated_delta_rule_prefill_amd as kda
    for n in (3000, 1024, 495, 1):
        x = ta.make(74, dtype, 4, 64, 64, [n], [n])
        args = dict(k_pe=x["k_pe"], scale=x["scale"])
        o, lse = kda.latent_attention(x["q"], x["k"], x["v"], **args)
        got = kda.latent_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], workspace=ws, **args)
        want = kda.latent_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], **args)
        for name in ("dq", "dk", "dv", "dk_pe"):
            assert torch.equal(got[name], want[name]), (n, name)
    ws = ones(b.latent_decode_workspace_bytes(256, 256, 32, 256, 64, dtype == "bf16"))
    for lens, new in (([300] * 40, [1] * 40), ([900, 70, 5], [20, 1, 1]), ([2000], [1])):
        x = td.make(75, dtype, 32, 256, 64, 16, lens, new)
        got, want = td.run(x, 256, workspace=ws), td.run(x, 256)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# 128 tiles of 64 rows and more (times heads): fp32 gradients that are not split
WHOLE = [([2100], [2100], 4), ([300, 1, 65, 129], [300, 1, 65, 129], 32), ([70, 40], [1000, 33], 32)]


@pytest.mark.parametrize("d,dr", [(128, 64), (128, 0), (64, 64), (64, 0)])
@pytest.mark.parametrize("lens_q,lens_k,H", WHOLE)
def test_fp32_gradients_of_batches_that_are_not_split(d, dr, lens_q, lens_k, H):
    x = ta.make(76, "f32", H, d, dr, lens_q, lens_k)
    ta.check_all("whole", x, ta.both(x, lens_q, lens_k, True), lens_q, lens_k, True)


@pytest.mark.parametrize("what", ["k", "v", "q", "d_o"])
def test_fp32_values_that_are_not_finite_in_batches_that_are_not_split(what):
    """NaN in a key reaches no row before it, NaN in a row no key behind it."""
    lens, H, bad = [300, 70], 32, 150
    x = ta.make(77, "f32", H, 128, 64, lens, lens)
    clean = dict(x)
    clean.update({n: x[n].clone() for n in ("q", "d_o")})
    if what in ("q", "d_o"):
        clean["q"][bad], clean["d_o"][bad] = 0.0, 0.0
    x[what] = x[what].clone()
    x[what][bad, :, 5] = float("nan")
    got = ta.both(x, lens, lens, True)
    want = ref.attention(clean["q"], clean["k"], clean["v"], clean["k_pe"], lens, lens, True, x["scale"], clean["d_o"])
    if what in ("k", "v"):
        names, parts = ("o", "lse", "dq"), (slice(0, bad), slice(300, 370))
    else:
        names, parts = ("dk", "dv", "dk_pe"), (slice(bad + 1, 370),)
    for n in names:
        for part in parts:
            ref.check(f"{what} {n}", got[n][part], want[n][0][part], want[n][1][part])


def test_fp32_is_fp32():
    """The element-wise bounds allow for errors that all have one sign.  In the
    norm they add like independent ones: a sum of n <= 400 terms is off by about
    sqrt(400) half steps of 2^-24, 1.2e-6, relative to its terms; a gradient has
    four such sums on its way (scores, g . v, delta, its own), 2.4e-6 together, and
    exponentials within 2^-22.  Operands cut to 16 bits would be off by 2^-17 each,
    1e-5 and more in all."""
    lens = [400, 90]
    for H, d, dr in ((2, 128, 64), (32, 64, 64)):            # split and whole
        x = ta.make(78, "f32", H, d, dr, lens, lens)
        got = ta.both(x, lens, lens, True)
        want = ref.attention(x["q"], x["k"], x["v"], x["k_pe"], lens, lens, True, x["scale"], x["d_o"])
        for n in ("o", "dq", "dk", "dv", "dk_pe"):
            rel = ref.check(f"fp32 {n}", got[n], *want[n])
            assert rel <= 4e-6, n
    for dl in (256, 512):
        x = td.make(79, "f32", 8, dl, 64, 16, [400, 90], [1, 3])
        o, _ = td.run(x, dl)
        assert ref.check("fp32 decode", o, *ref.decode(x["q"], x["cache"], x["table"], [400, 90], [1, 3], dl,
                                                        x["scale"])[0]) <= 4e-6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,new", [
    ([(97 * i) % 400 + 1 for i in range(40)], [1] * 40),     # 40 row tiles, joined row by row
    ([(13 * i) % 90 for i in range(300)], [1] * 300),        # more row tiles than workgroups
    ([900, 40, 200], [130, 40, 3]),                          # tiles of 64 rows, over 32 of them
])
def test_decode_of_512_channels_in_many_row_tiles(dtype, lens, new):
    x = td.make(80, dtype, 32, 512, 64, 16, lens, new)
    td.check(f"{len(lens)} sequences", x, 512, lens, new)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Tk", [(0, 0), (0, 70), (70, 0), (1, 0)])
@pytest.mark.parametrize("packed", [True, False])
def test_no_queries_or_no_keys(dtype, T, Tk, packed):
    import gated_delta_rule_prefill_amd as kda
    x = ta.make(81, dtype, 3, 128, 64, [T], [Tk])
    args = dict(k_pe=x["k_pe"], scale=x["scale"])
    if packed:
        args.update(cu_seqlens=ta.offsets([T]), cu_seqlens_k=ta.offsets([Tk]))
    o, lse = kda.latent_attention(x["q"], x["k"], x["v"], **args)
    g = kda.latent_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], **args)
    assert o.shape == (T, 3, 128) and (o == 0).all() and torch.isneginf(lse).all()
    for n, rows in (("dq", T), ("dk", Tk), ("dv", Tk), ("dk_pe", Tk)):
        assert g[n].shape[0] == rows and (g[n] == 0).all(), n


def test_no_tokens_in_the_paged_and_rotary_calls():
    import gated_delta_rule_prefill_amd as kda
    x = td.make(82, "bf16", 4, 256, 64, 16, [20, 5], [0, 0])
    before = x["cache"].clone()
    c = torch.zeros(0, 320, device="cuda", dtype=torch.bfloat16)
    for cu in (x["cu"], None):
        o, lse = td.run(x, 256, cu_seqlens=cu)
        assert o.shape == (0, 4, 256) and lse.shape == (0, 4)
        kda.latent_append(x["cache"], c[:, :256], x["table"], x["seq_lens"], k_pe=c[:, 256:], cu_seqlens=cu, c_out=True)
    assert torch.equal(x["cache"].view(torch.int16), before.view(torch.int16))
    freq, _ = kda.rotary_frequencies(64, device="cuda")
    assert kda.rotary(x["q"][..., :64], torch.zeros(0, dtype=torch.int32, device="cuda"), freq).shape == (0, 4, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_keys_and_values_that_the_heads_share(dtype):
    """Keys and values broadcast over the heads (stride 0), queries too: as dense copies."""
    import gated_delta_rule_prefill_amd as kda
    lens, H = [70, 200], 4
    x = ta.make(83, dtype, H, 128, 64, lens, lens)
    k, v = x["k"][:, :1].expand(-1, H, -1), x["v"][:, :1].expand(-1, H, -1)
    q = x["q"][:1, :1].expand(270, H, -1)
    args = dict(k_pe=x["k_pe"][:1].expand(270, -1), cu_seqlens=ta.offsets(lens), scale=x["scale"])
    dense = dict(args, k_pe=args["k_pe"].contiguous())
    o, lse = kda.latent_attention(q, k, v, **args)
    want = kda.latent_attention(q.contiguous(), k.contiguous(), v.contiguous(), **dense)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    got = kda.latent_attention_backward(q, k, v, o, lse, x["d_o"], **args)
    want = kda.latent_attention_backward(q.contiguous(), k.contiguous(), v.contiguous(), o, lse, x["d_o"], **dense)
    for n in got:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [5, 32])
def test_paged_offsets_that_start_late(dtype, H):
    """New tokens behind rows of no sequence, in decode and in append."""
    import gated_delta_rule_prefill_amd as kda
    lens, new, first = [150, 20], [30, 2], 7
    x = td.make(84, dtype, H, 256, 64, 16, lens, new, poison=False)
    want = td.run(x, 256)
    y = dict(x, q=torch.cat([x["q"][:first] * float("nan"), x["q"]]), cu=x["cu"] + first)
    out = torch.full((39, H, 256), 7.0, dtype=td.DT[dtype], device="cuda")
    lse = torch.full((39, H), 7.0, device="cuda")
    td.run(y, 256, out=out, lse=lse)
    assert (out[:first] == 7.0).all() and (lse[:first] == 7.0).all()
    wo, wl = ref.decode(x["q"], x["cache"], x["table"], lens, new, 256, x["scale"])
    ref.check("late o", out[first:], *wo)
    ref.check("late lse", lse[first:], *wl)
    ref.check("o", want[0], *wo)
    c = torch.randn(32, 320, device="cuda").to(td.DT[dtype])
    caches = [x["cache"].clone() for _ in range(2)]
    kda.latent_append(caches[0], c[:, :256], x["table"], x["seq_lens"], k_pe=c[:, 256:], cu_seqlens=x["cu"])
    late = torch.cat([c[:first], c])
    kda.latent_append(caches[1], late[:, :256], x["table"], x["seq_lens"], k_pe=late[:, 256:], cu_seqlens=y["cu"])
    assert torch.equal(caches[0], caches[1])
