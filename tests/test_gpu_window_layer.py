"""A window-attention layer as it is used: norm and rotation, attention and both
gradients over a training batch; prompts in pieces, then single tokens from a
captured graph, over a paged cache whose left pages are given back.  Against the
whole layer in float64.

Tolerances, of the relative L2 error.  An input of unit normal channels leaves the
norm as such; a rounded element is off by u (bf16 2^-8, fp32 work by 1e-4, see
window_reference.py), so a score, scale sum |q k| = 5 for 64 channels, by at most
2 u 5 = 10 u, and a weight by as much relatively.  An output takes the weights'
error and three roundings (weights, output, and the values it is compared on):
13 u.  A gradient takes it twice (weights; gradient of the scores through o), and
six roundings (queries and keys, weights, output, gradient of the scores, gradient
of queries and keys, gradient of the inputs): 26 u.  The weight of a channel is
within [0.5, 1.5] and only moves the scale.
"""
import pytest
import torch

import window_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 1e-4}
H, HK, D, DR = 6, 2, 64, 32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(seed, dtype, lens):
    import gated_delta_rule_prefill_amd as kda
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    return dict(qkv=torch.randn(T, H + 2 * HK, D, generator=g).to(DT[dtype]).cuda(),
                d_o=torch.randn(T, H, D, generator=g).to(DT[dtype]).cuda(),
                w=[(torch.rand(D, generator=g) + 0.5).cuda() for _ in range(2)],
                pos=torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda(),
                f=kda.rotary_frequencies(DR, device="cuda")[0])


def split(qkv):
    return qkv[:, :H], qkv[:, H:H + HK], qkv[:, H + HK:]


def turn(x, pos, f):
    """x with its first DR channels turned, differentiable."""
    ang = (pos.double()[:, None] * f.double()[None])[:, None]
    a, b, rest = x[..., :DR // 2], x[..., DR // 2:DR], x[..., DR:]
    return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin(), rest], dim=-1)


def layer64(x, lens, window, sinks):
    """(o, leaves): the layer in float64, its leaves qkv and the weights."""
    qkv = x["qkv"].double().cpu().requires_grad_()
    w = [y.double().cpu().requires_grad_() for y in x["w"]]
    pos, f = x["pos"].cpu(), x["f"].cpu()
    q, k, v = split(qkv)
    q, k = (turn(y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * z, pos, f) for y, z in ((q, w[0]), (k, w[1])))
    out, a = [], 0
    for n in lens:
        ks, vs = (y[a:a + n].repeat_interleave(H // HK, dim=1).transpose(0, 1) for y in (k, v))
        z = q[a:a + n].transpose(0, 1) @ ks.transpose(1, 2) * D ** -0.5
        z = z.masked_fill(~ref.sees(n, n, window, sinks)[None], -torch.inf)
        out.append((z.softmax(-1) @ vs).transpose(0, 1))
        a += n
    return torch.cat(out), [qkv, *w]


def close(name, got, want, tol):
    err = float((got.double().cpu() - want).norm() / want.norm())
    print(f"[layer] {name}: rel-L2 {err:.2e} (tolerance {tol:.1e})", flush=True)
    assert err <= tol, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,window,sinks", [([300, 1, 77], 50, 4), ([2100], 400, 64), ([40, 64, 65], 1000, 0)])
def test_training_step(dtype, lens, window, sinks):
    import gated_delta_rule_prefill_amd as kda
    x = make(71, dtype, lens)
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0)], dtype=torch.int32, device="cuda")
    q, k, v = split(x["qkv"])
    norm = dict(q_weight=x["w"][0], k_weight=x["w"][1], positions=x["pos"], inv_freq=x["f"])
    yq, yk = kda.qk_norm_rotary(q, k, **norm)
    args = dict(window=window, sinks=sinks, cu_seqlens=cu)
    o, lse = kda.window_attention(yq, yk, v, **args)
    grad = torch.empty_like(x["qkv"])       # the gradient of the projection, all of it written
    gq, gk, gv = split(grad)
    g = kda.window_attention_backward(yq, yk, v, o, lse, x["d_o"], dk=gk, dv=gv, **args)
    gq.copy_(g["dq"])
    n = kda.qk_norm_rotary_backward(q, k, gq, gk, dq=gq, dk=gk, **norm)
    torch.cuda.synchronize()
    want, leaves = layer64(x, lens, window, sinks)
    want.backward(x["d_o"].double().cpu())
    close("o", o, want.detach(), 13 * U[dtype])
    for name, got, leaf in (("dqkv", grad, leaves[0]), ("dq_weight", n["dq_weight"], leaves[1]),
                            ("dk_weight", n["dk_weight"], leaves[2])):
        close(name, got, leaf.grad, 26 * U[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving(dtype):
    """Three requests of other lengths: the first piece of a prompt through the
    packed attention, its second over the cache, then single tokens from a graph."""
    import gated_delta_rule_prefill_amd as kda
    window, sinks, page, steps = 70, 4, 16, 9
    first, second = [130, 5, 64], [37, 1, 70]
    lens = [a + b + steps for a, b in zip(first, second)]
    x = make(72, dtype, lens)
    want = layer64(x, lens, window, sinks)[0].detach()
    at = [0, lens[0], lens[0] + lens[1]]
    pages = [-(-n // page) for n in lens]
    P = sum(pages) + 2
    # heads before rows in a page, keys and values in one tensor
    pool = torch.full((2, P, HK, page, D), float("nan"), dtype=DT[dtype], device="cuda")
    kc, vc = (pool[i].transpose(1, 2) for i in range(2))
    order = torch.randperm(P, generator=torch.Generator().manual_seed(5)).int()
    table = torch.full((3, max(pages)), -1, dtype=torch.int32)
    for s, n in enumerate(pages):
        table[s, :n] = order[sum(pages[:s]):sum(pages[:s]) + n]
    table = table.cuda()
    seq_lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    norm = dict(norm_weight=x["w"][1], inv_freq=x["f"])
    out = torch.zeros_like(want)

    def step(done, new, decode):
        rows = torch.cat([torch.arange(a + d, a + d + n) for a, d, n in zip(at, done, new)]).cuda()
        cu = torch.tensor([0, *torch.tensor(new).cumsum(0)], dtype=torch.int32, device="cuda")
        q, k, v = split(x["qkv"][rows])
        seq_lens.copy_(torch.tensor([d + n for d, n in zip(done, new)], dtype=torch.int32))
        yq, _ = kda.qk_norm_rotary(q, None, q_weight=x["w"][0], positions=x["pos"][rows], inv_freq=x["f"])
        yk = kda.kv_append(kc, vc, k, v, table, seq_lens, cu_seqlens=cu, k_out=True, **norm)
        if decode:
            o, _ = kda.window_decode(yq, kc, vc, table, seq_lens, window=window, sinks=sinks, cu_seqlens=cu)
        else:
            o, _ = kda.window_attention(yq, yk, v, window=window, sinks=sinks, cu_seqlens=cu)
        out[rows.cpu()] = o.double().cpu()

    step([0, 0, 0], first, False)
    step(first, second, True)
    # the pages that every later token's window has left are given back and overwritten
    for s in range(3):
        left = first[s] + second[s] + 1 - window
        for j in range(1, pages[s]):
            if (j + 1) * page <= left:
                pool[:, int(table[s, j])] = float("inf")
                table[s, j] = -1
    # one token a step: a captured graph that reads its tokens from fixed tensors
    qkv, pos = torch.empty(3, H + 2 * HK, D, dtype=DT[dtype], device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.empty(kda.window_decode_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty(3, H, D, dtype=DT[dtype], device="cuda"), torch.empty(3, H, device="cuda")
    yq = torch.empty(3, H, D, dtype=DT[dtype], device="cuda")

    def token():
        q, k, v = split(qkv)
        kda.qk_norm_rotary(q, None, q_weight=x["w"][0], positions=pos, inv_freq=x["f"], q_out=yq)
        kda.kv_append(kc, vc, k, v, table, seq_lens, **norm)
        kda.window_decode(yq, kc, vc, table, seq_lens, window=window, sinks=sinks, out=o, lse=lse, workspace=ws)

    graph = None
    for i in range(steps):
        now = [a + b + i for a, b in zip(first, second)]
        rows = torch.tensor([a + n for a, n in zip(at, now)]).cuda()
        qkv.copy_(x["qkv"][rows])
        pos.copy_(x["pos"][rows])
        seq_lens.copy_(torch.tensor([n + 1 for n in now], dtype=torch.int32))
        if i < 2:
            token()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    token()
            graph.replay()
        torch.cuda.synchronize()
        out[rows.cpu()] = o.double().cpu()
    close("o", out, want, 13 * U[dtype])
