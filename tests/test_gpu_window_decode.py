"""Window attention over a paged cache, and the cache's writes, against their
definitions in float64, element by element."""
import pytest
import torch

import window_reference as ref
from test_gpu_guards import PATTERN, Guarded, _check

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def offsets(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def make(seed, dtype, H, Hk, d, page, lens, new, poison=True, behind=0):
    """A pool whose pages lie in random order; rows behind a sequence's end and
    free pages hold NaN (nothing of them may reach a result)."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-m // page) for m in lens]
    P = sum(used) + 3
    order = torch.randperm(P, generator=g)
    table = torch.full((len(lens), max(1, max(used))), -1, dtype=torch.int32)
    k, v = (torch.full((P, page, Hk, d), float("nan") if poison else 0.0) for _ in range(2))
    at = 0
    for s, (m, u) in enumerate(zip(lens, used)):
        table[s, :u] = order[at:at + u].int()
        for cache in (k, v):
            rows = torch.full((u * page, Hk, d), float("nan") if poison else 0.0)
            rows[:m] = torch.randn(m, Hk, d, generator=g)
            cache[order[at:at + u]] = rows.reshape(u, page, Hk, d)
        at += u
    q = torch.randn(sum(new) + behind, H, d, generator=g)
    return dict(q=q.to(DT[dtype]).cuda(), k=k.to(DT[dtype]).cuda(), v=v.to(DT[dtype]).cuda(), table=table.cuda(),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), cu=offsets(new))


def run(x, window, sinks, **kw):
    import gated_delta_rule_prefill_amd as kda
    kw.setdefault("cu_seqlens", x["cu"])
    return kda.window_decode(x["q"], x["k"], x["v"], x["table"], x["seq_lens"], window=window, sinks=sinks, **kw)


def check(label, x, lens, new, window, sinks, **kw):
    o, lse = run(x, window, sinks, **kw)
    torch.cuda.synchronize()
    (wo, eo), (wl, el) = ref.decode(x["q"], x["k"], x["v"], x["table"], lens, new, window, sinks)
    n = sum(new)
    ref.check(f"{label} o", o[:n], wo[:n], eo[:n])
    ref.check(f"{label} lse", lse[:n], wl[:n], el[:n])
    return o, lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,d", [(1, 1, 128), (8, 2, 64), (20, 1, 128), (32, 8, 64), (6, 3, 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 4), (1000, 64)])
def test_single_tokens(dtype, H, Hk, d, window, sinks):
    lens = [1, 64, 65, 0, 300, 17, 700]
    x = make(31, dtype, H, Hk, d, 16, lens, [1] * 7)
    check(f"{dtype} {H}/{Hk} {d} W={window}", x, lens, [1] * 7, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 7, 48, 64, 100, 128])
def test_page_sizes_and_several_tokens(dtype, page):
    lens, new = [40, 3, 200, 129, 64], [3, 3, 1, 0, 7]
    x = make(32, dtype, 8, 2, 128, page, lens, new)
    check(f"{dtype} page {page}", x, lens, new, 60, 4)
    check(f"{dtype} page {page}, one key and the sinks", x, lens, new, 1, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (33, 4), (500, 64)])
def test_chunks_of_new_tokens(dtype, d, window, sinks):
    """Many rows per sequence; a whole prompt (no prefix); more new tokens than
    the cache is said to hold (rows that see nothing)."""
    lens, new = [460, 70, 10, 33], [165, 70, 14, 1]
    x = make(33, dtype, 8, 2, d, 64, lens, new)
    check(f"{dtype} chunks", x, lens, new, window, sinks)


def test_equal_rows():
    lens = [100, 40, 77]
    for each in (1, 2, 30):
        x = make(34, "bf16", 16, 4, 128, 64, lens, [each] * 3)
        check("equal rows", x, lens, [each] * 3, 20, 2, cu_seqlens=None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_long_sequence(dtype):
    """Its keys split over workgroups, the parts joined."""
    lens = [9000]
    x = make(35, dtype, 32, 8, 128, 64, lens, [1])
    check("window of 4,096", x, lens, [1], 4096, 4)
    check("whole cache", x, lens, [1], 2 ** 31 - 1, 0)


@pytest.mark.parametrize("H,Hk", [(4, 2), (24, 3)])
def test_many_sequences(H, Hk):
    """More sequences than a workgroup has threads."""
    lens = [(13 * i) % 90 for i in range(1100)]
    new = [1 if i % 7 else 0 for i in range(1100)]
    x = make(36, "bf16", H, Hk, 64, 16, lens, new)
    check(f"1100 sequences {H}/{Hk}", x, lens, new, 30, 4)


@pytest.mark.parametrize("new", [[1] * 4, [70] * 4])
def test_bad_pages_and_lengths(new):
    """Pages outside the pool count as absent; a length beyond the table's room
    is clamped to it, a negative one to zero."""
    lens = [100, 100, 90, 74]
    x = make(37, "bf16", 8, 2, 128, 16, lens, new)
    x["table"][0, 2] = -1
    x["table"][1, 0] = x["k"].shape[0]
    x["table"][1, 6] = 2 ** 31 - 1
    x["table"][2, :] = -5
    check("bad pages", x, lens, new, 70, 4)
    x = make(38, "bf16", 8, 2, 128, 16, [112] * 4, new, poison=False)
    x["seq_lens"][0] = 2 ** 31 - 1
    x["seq_lens"][1] = -3
    check("bad lengths", x, [2 ** 31 - 1, -3, 112, 112], new, 70, 4)


@pytest.mark.parametrize("new", [1, 60])
def test_pages_that_the_window_has_left(new):
    """Their table entries given back, those of the sinks kept: the same results."""
    lens, page, window, sinks = [700, 90], 16, 100, 20
    x = make(39, "bf16", 8, 2, 128, page, lens, [new] * 2)
    want = check("all pages", x, lens, [new] * 2, window, sinks)
    for s, m in enumerate(lens):
        first = max(0, m - new - window + 1) // page
        for j in range(-(-sinks // page), first):
            x["table"][s, j] = -1
    got = run(x, window, sinks)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [[7, 3], [60, 40]])
@pytest.mark.parametrize("what,value", [("k", "nan"), ("v", "nan"), ("v", "-inf"), ("k", "inf")])
def test_hidden_rows_that_are_not_finite(dtype, new, what, value):
    """Of several new tokens those that do not see a row with NaN or Inf are
    clean, before it or beyond its window."""
    lens, window, sinks = [150, 90], 30, 4
    x = make(40, dtype, 8, 2, 128, 16, lens, new, poison=False)
    (wo, eo), (wl, el) = ref.decode(x["q"], x["k"], x["v"], x["table"], lens, new, window, sinks)
    t = 0
    hidden = torch.ones(sum(new), dtype=torch.bool)
    for s, (m, n) in enumerate(zip(lens, new)):
        for bad in (m - n // 2, m - n + 1 - window):    # a new token, and one that the window leaves
            x[what][x["table"][s, bad // 16].long(), bad % 16, :, 7] = float(value)
            p = torch.arange(m - n, m)
            hidden[t:t + n] &= (p < bad) | (p - bad >= window)
        t += n
    o, lse = run(x, window, sinks)
    h = hidden.cuda()
    assert hidden.any() and not hidden.all()
    ref.check(f"hidden {what} {value} o", o[h], wo[hidden], eo[hidden])
    ref.check(f"hidden {what} {value} lse", lse[h], wl[hidden], el[hidden])
    assert not torch.isfinite(o[~h].float()).all(dim=-1).any() or what == "k"


@pytest.mark.parametrize("layout", ["heads first", "halves", "padded"])
def test_cache_layouts(layout):
    lens, new = [300, 17, 64], [1, 3, 2]
    x = make(41, "bf16", 8, 2, 128, 16, lens, new)
    want = run(x, 40, 4)
    P, page, Hk, d = x["k"].shape
    if layout == "heads first":
        x["k"], x["v"] = (x[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "kv")
    elif layout == "halves":
        both = torch.stack([x["k"], x["v"]], dim=1)
        x["k"], x["v"] = both[:, 0], both[:, 1]
    else:
        wide = torch.full((2, P, page + 1, Hk + 1, d + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[0, :, :page, :Hk, :d], wide[1, :, :page, :Hk, :d] = x["k"], x["v"]
        x["k"], x["v"] = wide[0, :, :page, :Hk, :d], wide[1, :, :page, :Hk, :d]
    got = run(x, 40, 4)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [[1, 1, 1], [70, 0, 3]])
def test_writes_stay_in_bounds(dtype, new):
    import gated_delta_rule_prefill_amd as kda
    lens, H, t = [300, 17, 64], 6, DT[dtype]
    x = make(42, dtype, H, 2, 64, 16, lens, new)
    T = sum(new)
    need = kda.window_decode_workspace_bytes(64)
    out = dict(o=Guarded((T, H, 64), t), lse=Guarded((T, H), torch.float32),
               ws=Guarded((need,), torch.uint8, init=torch.full((need,), 255, dtype=torch.uint8, device="cuda")))
    check("guarded", x, lens, new, 50, 4, out=out["o"].t, lse=out["lse"].t, workspace=out["ws"].t)
    _check(out, f"window decode {dtype}")


@pytest.mark.parametrize("each", [1, 40])
def test_rows_behind_the_last_sequence_are_left(each):
    lens, new = [100, 50], [each, each]
    x = make(43, "bf16", 8, 2, 128, 16, lens, new, behind=9)
    out = torch.full((2 * each + 9, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2 * each + 9, 8), 7.0, device="cuda")
    check("behind", x, lens, new, 30, 4, out=out, lse=lse)
    assert (out[2 * each:] == 7.0).all() and (lse[2 * each:] == 7.0).all()


def test_large_cache():
    """Rows beyond 2^31 elements from the cache's start."""
    import gated_delta_rule_prefill_amd as kda
    page, Hk, d, H = 64, 8, 128, 16
    P = (1 << 31) // (page * Hk * d) + 40
    k, v = (torch.empty(P, page, Hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[P - 1, 0, P - 7, P - 2]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(44)
    for p in (P - 1, 0, P - 7, P - 2):
        for cache in (k, v):
            cache[p] = torch.randn(page, Hk, d, generator=g).bfloat16().cuda()
    lens = [250]
    for new in ([1], [90]):
        x = dict(q=torch.randn(new[0], H, d, generator=g).bfloat16().cuda(), k=k, v=v, table=table,
                 seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), cu=offsets(new))
        check(f"large, {new}", x, lens, new, 150, 4)
    rows = torch.randn(2, 3, Hk, d, generator=g).bfloat16().cuda()
    kda.kv_append(k, v, rows[0], rows[1], table, torch.tensor([66], dtype=torch.int32, device="cuda"),
                  cu_seqlens=offsets([3]))
    assert torch.equal(k[P - 1, 63], rows[0, 0]) and torch.equal(v[0, :2], rows[1, 1:])


def test_graph_replays_match_eager():
    """A step (append, then attention) captured once and replayed on new tokens and lengths."""
    import gated_delta_rule_prefill_amd as kda
    H, Hk, d, page, n = 8, 2, 128, 16, 5
    g = torch.Generator().manual_seed(45)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    table = torch.randperm(40, generator=g).int().reshape(n, 8).cuda()
    caches = [r(40, page, Hk, d) for _ in range(2)]
    freq, _ = kda.rotary_frequencies(d, device="cuda")
    w = torch.rand(d, generator=g).cuda() + 0.5
    s = dict(q=r(n, H, d), kv=r(n, 2 * Hk, d), lens=torch.tensor([1, 20, 33, 90, 127], dtype=torch.int32, device="cuda"))

    def step(kc, vc):
        kda.kv_append(kc, vc, s["kv"][:, :Hk], s["kv"][:, Hk:], table, s["lens"], norm_weight=w, inv_freq=freq)
        return kda.window_decode(s["q"], kc, vc, table, s["lens"], window=40, sinks=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*[c.clone() for c in caches])
    torch.cuda.current_stream().wait_stream(side)
    mine = [c.clone() for c in caches]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*mine)
    for i in range(4):
        s["q"].copy_(r(n, H, d))
        s["kv"].copy_(r(n, 2 * Hk, d))
        want = step(*caches)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(list(outs) + mine, list(want) + caches):
            assert torch.equal(a, b), i
        s["lens"].add_(torch.tensor([1, 1, 1, 1, 0], dtype=torch.int32, device="cuda"))


def test_calls_at_the_same_time():
    """Split decodes on two streams at once, each with its own workspace, give what they give alone."""
    lens = [5000]
    xs = [make(46 + i, "bf16", 16, 4, 128, 64, lens, [1]) for i in range(2)]
    want = [run(x, 4096, 4) for x in xs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = [run(x, 4096, 4, stream=st) for x, st in zip(xs, (None, side))]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# -- the cache's writes ------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,start,dr,interleaved", [(128, 0, 128, False), (128, 64, 64, True), (64, 0, 32, False),
                                                    (64, 3, 26, False), (128, 1, 30, True), (64, 0, 0, False)])
@pytest.mark.parametrize("normed", [True, False])
def test_append(dtype, d, start, dr, interleaved, normed):
    """New tokens' rows by the formula, every other row of the cache as it was."""
    import gated_delta_rule_prefill_amd as kda
    lens, new, page, Hk, t = [40, 3, 200, 129, 5], [3, 3, 61, 0, 7], 16, 3, DT[dtype]
    x = make(48, dtype, Hk, Hk, d, page, lens, [1] * 5)
    g = torch.Generator().manual_seed(49)
    T = sum(new) + 4
    kv = torch.randn(T, 2 * Hk, d, generator=g).to(t).cuda()
    w = (torch.rand(d, generator=g) + 0.5).cuda() if normed else None
    freq, _ = kda.rotary_frequencies(dr, device="cuda") if dr else (None, 1.0)
    k0, v0 = x["k"].clone(), x["v"].clone()
    k_out = torch.full((T, Hk, d), 7.0, dtype=t, device="cuda")
    kda.kv_append(x["k"], x["v"], kv[:, :Hk], kv[:, Hk:], x["table"], x["seq_lens"], cu_seqlens=offsets(new),
                  norm_weight=w, eps=1e-5, inv_freq=freq, start=start, interleaved=interleaved, mscale=1.25, k_out=k_out)
    at, place = 0, []
    for s, (m, n) in enumerate(zip(lens, new)):
        place += [(s, m - n + i) for i in range(n)]
    n = sum(new)
    pos = torch.tensor([p for _, p in place], dtype=torch.int32)
    want, bound = ref.norm(kv[:n, :Hk], w, pos, freq, start, interleaved, 1e-5, 1.25, normalise=normed)
    ref.check("k_out", k_out[:n], want, bound)
    assert (k_out[n:] == 7.0).all()
    touched = torch.zeros(x["k"].shape[:2], dtype=torch.bool)
    for i, (s, p) in enumerate(place):
        if p >= 0:
            page_at = int(x["table"][s, p // page])
            assert torch.equal(x["k"][page_at, p % page], k_out[i]) and torch.equal(x["v"][page_at, p % page], kv[i, Hk:])
            touched[page_at, p % page] = True
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    rest = (~touched).cuda()
    assert same(x["k"][rest], k0[rest]) and same(x["v"][rest], v0[rest])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_writes_stay_in_bounds(dtype):
    import gated_delta_rule_prefill_amd as kda
    t, d, page, Hk, lens, new = DT[dtype], 64, 16, 2, [20, 5], [7, 5]
    T = sum(new)
    g = torch.Generator().manual_seed(50)
    kv = torch.randn(T, 2 * Hk, d, generator=g).to(t).cuda()
    table = torch.tensor([[2, 0], [1, -1]], dtype=torch.int32, device="cuda")
    freq, _ = kda.rotary_frequencies(32, device="cuda")
    out = dict(k=Guarded((3, page, Hk, d), t), v=Guarded((3, page, Hk, d), t), k_out=Guarded((T, Hk, d), t))
    kda.kv_append(out["k"].t, out["v"].t, kv[:, :Hk], kv[:, Hk:], table,
                  torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_seqlens=offsets(new), inv_freq=freq, start=16,
                  k_out=out["k_out"].t)
    _check(out, f"kv append {dtype}")
    rows = [16 * (2 if p < 16 else 0) + p % 16 for p in range(13, 20)] + [16 + p for p in range(5)]
    for name in "kv":
        written = (out[name].t.view(torch.uint8) != PATTERN).reshape(3 * page, -1).any(dim=1).nonzero().flatten().tolist()
        assert written == sorted(rows)


def test_append_bad_pages_and_lengths():
    """Tokens without a place are not written, their keys still go to k_out."""
    import gated_delta_rule_prefill_amd as kda
    Hk, d, page = 2, 64, 16
    k, v = (torch.full((4, page, Hk, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[4, 1], [-1, 2 ** 31 - 1], [0, 2], [3, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 20, 3, -4], dtype=torch.int32, device="cuda")
    kv = torch.randn(4 * 6, 2 * Hk, d).bfloat16().cuda()
    k_out = kda.kv_append(k, v, kv[:, :Hk], kv[:, Hk:], table, lens, k_out=True)
    assert torch.equal(k_out, kv[:, :Hk])
    want = torch.full_like(k, 7.0)
    want[1, :4] = kv[2:6, :Hk]          # positions 16 .. 19 of sequence 0; 14 and 15 lie in a page outside the pool
    want[0, :3] = kv[15:18, :Hk]        # sequence 2 holds 3 tokens: the first 3 of 6 new ones have no place
    assert torch.equal(k, want)


def test_append_single_tokens_and_many_sequences():
    import gated_delta_rule_prefill_amd as kda
    n, Hk, d, page = 1500, 1, 64, 4
    table = torch.randperm(2 * n).int().reshape(n, 2).cuda()
    lens = torch.randint(1, 9, (n,), dtype=torch.int32).cuda()
    k, v = (torch.zeros(2 * n, page, Hk, d, device="cuda") for _ in range(2))
    kv = torch.randn(n, 2, d, device="cuda")
    for cu in (None, torch.arange(n + 1, dtype=torch.int32, device="cuda")):
        kda.kv_append(k.zero_(), v.zero_(), kv[:, :1], kv[:, 1:], table, lens, cu_seqlens=cu)
        p = (lens - 1).long()
        pages = table[torch.arange(n, device="cuda"), p // page].long()
        assert torch.equal(k[pages, p % page], kv[:, :1]) and torch.equal(v[pages, p % page], kv[:, 1:])
        assert int((k != 0).any(-1).sum()) == n
