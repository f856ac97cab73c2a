"""The window operators at the calls their documentation allows and a model seldom
makes: grids of more than one row, groups wider than a tile of rows, inputs that heads
or tokens share, pages that sequences share, offsets that start late, workspaces that
hold anything or that captured graphs share."""
import pytest
import torch

import test_gpu_window_attention as ta
import test_gpu_window_decode as td
import window_reference as ref

pytestmark = pytest.mark.gpu
DT = ta.DT


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("packed", [False, True])
def test_grids_of_more_than_one_row(dtype, packed):
    """70,000 sequences of one token, a workgroup each: o = v, dv = d_o, no other gradient."""
    N, d = 70000, 64
    x = ta.make(91, dtype, 1, 1, d, [N], [N])
    import gated_delta_rule_prefill_amd as kda
    args = dict(window=3, sinks=1)
    if packed:
        args["cu_seqlens"] = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    else:
        args["num_seqs"] = N
    o, lse = kda.window_attention(x["q"], x["k"], x["v"], **args)
    g = kda.window_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], **args)
    torch.cuda.synchronize()
    # Not equal to the bit: with the score's maximum rounded once and the score itself inside a
    # multiply-add the weight is 2^e, |e| <= 2^-24 |z log2 e|, and o = (2^e v) (1 / 2^e), three
    # roundings; dv takes its weight from the rounded lse.  window_reference.py has the bounds.
    u, uw = ref.U[DT[dtype]], ref.U[DT[dtype]] if dtype == "bf16" else 0.0
    for got, want in ((o, x["v"]), (g["dv"], x["d_o"])):
        assert ((got.double() - want.double()).abs() <= (uw + u + ref.SLACK) * want.double().abs()).all()
    q, k, v, d_o = (x[n].double() for n in ("q", "k", "v", "d_o"))
    z = (q * k).sum(-1) * d ** -0.5
    assert ((lse[:, 0].double() - z[:, 0]).abs() <= ref.SLACK + 2.0 ** -22 * z[:, 0].abs()).all()
    # dz = d_o . v - delta: 0 but for the error of o in delta and that of the sums
    mag = (d_o.abs() * v.abs()).sum(-1, keepdim=True)
    for name, other in (("dq", k), ("dk", q)):
        assert (g[name].double().abs() <= (uw + u + 3 * ref.SLACK) * mag * other.abs() * d ** -0.5).all(), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,lens", [(200, 1, [9, 1, 30]), (260, 2, [5, 17])])
def test_groups_wider_than_a_tile(dtype, H, Hk, lens):
    x = ta.make(92, dtype, H, Hk, 64, lens, lens)
    ta.check_all(f"{H}/{Hk}", x, ta.both(x, lens, lens, 7, 2), lens, lens, 7, 2)
    y = td.make(93, dtype, H, Hk, 64, 16, [40, 9, 100], [1, 1, 1])
    td.check(f"{H}/{Hk}", y, [40, 9, 100], [1, 1, 1], 30, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_inputs_that_heads_and_tokens_share(dtype):
    """Strides of 0, and one tensor as keys and values, give what copies give."""
    lens, H, Hk, d = [70, 33], 8, 4, 64
    T = sum(lens)
    x = ta.make(94, dtype, H, Hk, d, lens, lens)
    shared = dict(q=x["q"][:1, :1].expand(T, H, d), k=x["k"][:, :1].expand(T, Hk, d), d_o=x["d_o"])
    for v in ("k", "v"):
        shared["v"] = shared["k"] if v == "k" else x["v"]
        got = ta.both(shared, lens, lens, 20, 3)
        want = ta.both({n: t.contiguous() for n, t in shared.items()}, lens, lens, 20, 3)
        assert all(torch.equal(got[n], want[n]) for n in want)
        ta.check_all(f"shared, {v} as values", shared, got, lens, lens, 20, 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 1, 40]])
def test_shared_and_repeated_pages(dtype, new):
    """Two sequences with the same first pages, and one whose page comes twice."""
    lens = [90, 80, 64]
    x = td.make(95, dtype, 8, 2, 64, 16, lens, new)
    table = x["table"]
    table[1, :3] = table[0, :3]
    table[2, 3] = table[2, 1]
    x["k"].nan_to_num_(nan=0.5)
    x["v"].nan_to_num_(nan=-0.5)
    td.check("shared pages", x, lens, new, 50, 4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [[1, 2, 1], [40, 1, 70]])
def test_paged_offsets_that_start_late(dtype, new):
    import gated_delta_rule_prefill_amd as kda
    lens, first, behind, T = [100, 50, 90], 5, 4, sum(new)
    x = td.make(96, dtype, 8, 2, 64, 16, lens, new, behind=first + behind)
    inner = dict(x, q=x["q"][first:first + T])
    x["q"][:first] = x["q"][first + T:] = float("nan")
    out = torch.full((T + first + behind, 8, 64), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T + first + behind, 8), 7.0, device="cuda")
    td.run(dict(x, cu=x["cu"] + first), 30, 4, out=out, lse=lse)
    torch.cuda.synchronize()
    (wo, eo), (wl, el) = ref.decode(inner["q"], x["k"], x["v"], x["table"], lens, new, 30, 4)
    part = slice(first, first + T)
    ref.check("late o", out[part], wo, eo)
    ref.check("late lse", lse[part], wl, el)
    for t in (out, lse):
        assert (t[:first] == 7.0).all() and (t[first + T:] == 7.0).all()
    # the cache's writes, with and without the rows around
    kv = torch.randn(T + first + behind, 4, 64, device="cuda").to(DT[dtype])
    kc, vc, kc2, vc2 = (torch.full_like(x["k"], 7.0) for _ in range(4))
    k_out = torch.full((T + first + behind, 2, 64), 7.0, dtype=DT[dtype], device="cuda")
    kda.kv_append(kc, vc, kv[:, :2], kv[:, 2:], x["table"], x["seq_lens"], cu_seqlens=x["cu"] + first, k_out=k_out)
    kda.kv_append(kc2, vc2, kv[part, :2], kv[part, 2:], x["table"], x["seq_lens"], cu_seqlens=x["cu"])
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2) and torch.equal(k_out[part], kv[part, :2])
    assert (k_out[:first] == 7.0).all() and (k_out[first + T:] == 7.0).all()


def ones(n):
    """A workspace whose every word is NaN, as bf16 and as fp32."""
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dirty_workspaces_change_nothing(dtype):
    import gated_delta_rule_prefill_amd as kda
    lens = [1500, 3, 0, 700]
    x = ta.make(97, dtype, 4, 2, 64, lens, lens)
    args = dict(window=50, sinks=9, cu_seqlens=ta.offsets(lens))
    o, lse = kda.window_attention(x["q"], x["k"], x["v"], **args)
    ws = [f(kda.window_attention_backward_workspace_bytes(sum(lens), 4, 4, 2, 64, 9))
          for f in (ones, lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda"))]
    a, b = (kda.window_attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], workspace=w, **args) for w in ws)
    assert all(torch.equal(a[n], b[n]) for n in a)
    y = td.make(98, dtype, 8, 2, 64, 16, [900, 3, 0], [1, 1, 1])
    n = kda.window_decode_workspace_bytes(64)
    a, b = (td.run(y, 800, 4, workspace=w) for w in (ones(n), torch.zeros(n, dtype=torch.uint8, device="cuda")))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    z = torch.randn(2, 300, 6, 64, device="cuda").to(DT[dtype])
    w = torch.rand(64, device="cuda")
    n = kda.qk_norm_rotary_backward_workspace_bytes(64)
    a, b = (kda.qk_norm_rotary_backward(z[0, :, :4], z[0, :, 4:], z[1, :, :4], z[1, :, 4:], q_weight=w, k_weight=w, workspace=s)
            for s in (ones(n), torch.zeros(n, dtype=torch.uint8, device="cuda")))
    assert all(torch.equal(a[m], b[m]) for m in a)


def test_two_graphs_with_one_workspace():
    """Captured decode calls of two layers, replayed one after the other while the
    lengths grow, against eager calls."""
    import gated_delta_rule_prefill_amd as kda
    ws = torch.empty(kda.window_decode_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    layers = [td.make(99 + i, "bf16", 8, 2, 128, 16, [700, 200, 50], [1, 1, 1], poison=False) for i in range(2)]
    outs = [(torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 8, device="cuda")) for _ in layers]
    graphs = []
    for x, (o, lse) in zip(layers, outs):
        td.run(x, 600, 4, out=o, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            td.run(x, 600, 4, out=o, lse=lse, workspace=ws)
        graphs.append(graph)
    for step in range(4):
        for x, (o, lse) in zip(layers, outs):
            x["seq_lens"] += 1
            x["q"].copy_(torch.randn_like(x["q"].float()))
            o.fill_(float("nan"))
        for _ in range(2):
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        for x, (o, lse) in zip(layers, outs):
            want = td.run(x, 600, 4)
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), step
