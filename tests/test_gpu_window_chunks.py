"""Chunks of new tokens in batches large enough for the forward kernel's paged form
(more than 512 row tiles of 16 rows over all key heads), against the definitions in
float64: the cases of test_gpu_window_decode.py, whose batches take the decode kernel."""
import pytest
import torch

import test_gpu_window_decode as td
import window_reference as ref
from test_gpu_guards import Guarded, _check

pytestmark = pytest.mark.gpu
DT = td.DT


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(seed, dtype, d, page, lens, new, H=40, Hk=40, **kw):
    assert (sum(new) * (H // Hk) // 16 + len(new)) * Hk > 512 and sum(new) * (H // Hk) > 16 * len(new)
    return td.make(seed, dtype, H, Hk, d, page, lens, new, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,d,page", [(40, 40, 64, 16), (40, 40, 128, 7), (32, 8, 64, 64), (24, 12, 128, 100), (18, 9, 64, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 4), (500, 64)])
def test_chunks(dtype, H, Hk, d, page, window, sinks):
    lens, new = [460, 70, 10, 333], [265, 70, 14, 150]      # in the third more new tokens than the cache holds
    x = make(101, dtype, d, page, lens, new, H, Hk)
    td.check(f"{dtype} {H}/{Hk} {d} page {page}", x, lens, new, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_rows(dtype):
    lens = [130, 40, 77, 200]
    x = make(102, dtype, 64, 64, lens, [60] * 4)
    td.check("equal rows", x, lens, [60] * 4, 20, 2, cu_seqlens=None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_pages_and_lengths(dtype):
    lens, new = [100, 100, 90, 74], [70] * 4
    x = make(103, dtype, 64, 16, lens, new)
    x["table"][0, 2] = -1
    x["table"][1, 0] = x["k"].shape[0]
    x["table"][1, 6] = 2 ** 31 - 1
    x["table"][2, :] = -5
    td.check("bad pages", x, lens, new, 70, 4)
    x = make(104, dtype, 64, 16, [112] * 4, new, poison=False)
    x["seq_lens"][0] = 2 ** 31 - 1
    x["seq_lens"][1] = -3
    td.check("bad lengths", x, [2 ** 31 - 1, -3, 112, 112], new, 70, 4)


def test_pages_that_the_window_has_left():
    lens, new, page, window, sinks = [700, 190], [150, 150], 16, 100, 20
    x = make(105, "bf16", 64, page, lens, new)
    want = td.check("all pages", x, lens, new, window, sinks)
    for s, (m, n) in enumerate(zip(lens, new)):
        for j in range(-(-sinks // page), max(0, m - n - window + 1) // page):
            x["table"][s, j] = -1
    got = td.run(x, window, sinks)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what,value", [("k", "nan"), ("v", "nan"), ("v", "-inf"), ("k", "inf")])
def test_hidden_rows_that_are_not_finite(dtype, what, value):
    lens, new, window, sinks = [350, 190], [160, 140], 30, 4
    x = make(106, dtype, 64, 16, lens, new, poison=False)
    (wo, eo), (wl, el) = ref.decode(x["q"], x["k"], x["v"], x["table"], lens, new, window, sinks)
    t, hidden = 0, torch.ones(sum(new), dtype=torch.bool)
    for s, (m, n) in enumerate(zip(lens, new)):
        for bad in (m - n // 2, m - n + 1 - window):    # a new token, and one that the window leaves
            x[what][x["table"][s, bad // 16].long(), bad % 16, :, 7] = float(value)
            p = torch.arange(m - n, m)
            hidden[t:t + n] &= (p < bad) | (p - bad >= window)
        t += n
    o, lse = td.run(x, window, sinks)
    h = hidden.cuda()
    assert hidden.any() and not hidden.all()
    ref.check(f"hidden {what} {value} o", o[h], wo[hidden], eo[hidden])
    ref.check(f"hidden {what} {value} lse", lse[h], wl[hidden], el[hidden])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_writes_stay_in_bounds_and_rows_behind_are_left(dtype):
    lens, new, first, behind = [200, 17, 264], [100, 10, 130], 3, 9
    T = sum(new)
    x = make(107, dtype, 64, 16, lens, new, behind=first + behind)
    out = dict(o=Guarded((T, 40, 64), DT[dtype]), lse=Guarded((T, 40), torch.float32))
    td.check("guarded", dict(x, q=x["q"][:T]), lens, new, 50, 4, out=out["o"].t, lse=out["lse"].t)
    _check(out, f"window chunks {dtype}")
    o = torch.full((T + first + behind, 40, 64), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T + first + behind, 40), 7.0, device="cuda")
    y = dict(x, q=torch.cat([x["q"][:1].expand(first, -1, -1) * float("nan"), x["q"][:T + behind]]), cu=x["cu"] + first)
    td.run(y, 50, 4, out=o, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(o[first:first + T], out["o"].t) and torch.equal(lse[first:first + T], out["lse"].t)
    for t in (o, lse):
        assert (t[:first] == 7.0).all() and (t[first + T:] == 7.0).all()


def test_large_cache():
    """Rows beyond 2^31 elements from the cache's start."""
    page, Hk, d, H = 64, 8, 128, 16
    P = (1 << 31) // (page * Hk * d) + 40
    k, v = (torch.empty(P, page, Hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = [P - 1, 0, P - 7, P - 2] + list(range(P // 2, P // 2 + 9))
    table = torch.tensor([pages], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(108)
    for p in pages:
        for cache in (k, v):
            cache[p] = torch.randn(page, Hk, d, generator=g).bfloat16().cuda()
    lens, new = [820], [600]
    x = dict(q=torch.randn(600, H, d, generator=g).bfloat16().cuda(), k=k, v=v, table=table,
             seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), cu=td.offsets(new))
    td.check("large", x, lens, new, 150, 4)


def test_graph_replays_match_eager():
    lens, new = [300, 150, 90], [100, 60, 60]
    x = make(109, "bf16", 64, 16, lens, new, poison=False)
    o, lse = torch.empty(220, 40, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(220, 40, device="cuda")
    td.run(x, 60, 4, out=o, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        td.run(x, 60, 4, out=o, lse=lse)
    for step in range(3):
        x["seq_lens"] -= 7
        x["q"].copy_(torch.randn_like(x["q"].float()))
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = td.run(x, 60, 4)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), step
