"""The norm and rotation of queries and keys, forwards and back, against the
definition in float64, element by element (bounds in window_reference.py)."""
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


def make(seed, dtype, T, H, Hk, d, dr, far=5000):
    import gated_delta_rule_prefill_amd as kda
    g = torch.Generator().manual_seed(seed)
    qkv, grad = (torch.randn(T, H + 2 * Hk, d, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    w = [(torch.rand(d, generator=g) + 0.5).cuda() for _ in range(2)]
    return dict(q=qkv[:, :H], k=qkv[:, H:H + Hk], dq_out=grad[:, :H], dk_out=grad[:, H:H + Hk], q_weight=w[0],
                k_weight=w[1], positions=torch.randint(0, far, (T,), generator=g, dtype=torch.int32).cuda() if dr else None,
                inv_freq=kda.rotary_frequencies(dr, device="cuda")[0] if dr else None)


def check(label, x, start=0, interleaved=False, eps=1e-6, mscale=1.0, keys=True, **kw):
    import gated_delta_rule_prefill_amd as kda
    args = {n: x[n] for n in ("q_weight", "k_weight", "positions", "inv_freq")}
    args.update(start=start, interleaved=interleaved, eps=eps, mscale=mscale)
    k, dk_out = (x["k"], x["dk_out"]) if keys else (None, None)
    if not keys:
        args["k_weight"] = None
    yq, yk = kda.qk_norm_rotary(x["q"], k, **args)
    g = kda.qk_norm_rotary_backward(x["q"], k, x["dq_out"], dk_out, **args)
    torch.cuda.synchronize()
    for name, y in (("q", yq), ("k", yk)):
        if y is None:
            assert g["dk"] is None and g["dk_weight"] is None
            continue
        rot = (x["positions"], x["inv_freq"], start, interleaved, eps, mscale)
        ref.check(f"{label} {name}", y, *ref.norm(x[name], x[f"{name}_weight"], *rot))
        dx, dw = ref.norm_backward(x[name], x[f"d{name}_out"], x[f"{name}_weight"], *rot)
        ref.check(f"{label} d{name}", g[f"d{name}"], *dx)
        if x[f"{name}_weight"] is None:
            assert g[f"d{name}_weight"] is None
        else:
            ref.check(f"{label} d{name}_weight", g[f"d{name}_weight"], *dw)
    return yq, yk, g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,start,dr", [(128, 0, 128), (128, 64, 64), (64, 0, 32), (256, 0, 256), (80, 16, 64), (96, 0, 96),
                                        (80, 3, 34), (6, 2, 4), (2, 0, 2), (250, 0, 250), (128, 0, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_shapes(dtype, d, start, dr, interleaved):
    for T, H, Hk in ((1, 1, 1), (37, 5, 2)):
        x = make(51, dtype, T, H, Hk, d, dr)
        check(f"{dtype} {d} [{start}, +{dr}) {interleaved}", x, start, interleaved, mscale=1.25)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tokens(dtype):
    """More tokens than the workgroups take at once; far positions."""
    x = make(52, dtype, 9001, 3, 2, 64, 64, far=2 ** 31 - 1)
    check(f"many {dtype}", x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_weights_or_keys(dtype):
    x = make(53, dtype, 70, 4, 2, 128, 64)
    check("no keys", x, keys=False)
    x["q_weight"] = None
    check("no q weight", x)
    x["k_weight"] = None
    check("no weights", x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,off", [(128, 0), (128, 1), (40, 3)])
def test_in_place_and_strides(dtype, d, off):
    """Parts of wider, unaligned tensors; forwards into the input, back into the
    output's gradient or the input, or into parts of one gradient."""
    import gated_delta_rule_prefill_amd as kda
    T, H, Hk = 33, 3, 2
    x = make(54, dtype, T, H, Hk, d, 32)
    args = {n: x[n] for n in ("q_weight", "k_weight", "positions", "inv_freq")}
    want = {}
    for n in "qk":
        rot = (x[f"{n}_weight"], x["positions"], x["inv_freq"], 0, False)
        want[n] = ref.norm(x[n], *rot)
        want["d" + n], want[f"d{n}_weight"] = ref.norm_backward(x[n], x[f"d{n}_out"], *rot)

    def part(t):
        wide = torch.full((T, t.shape[1] + 1, d + 5), 7.0, dtype=t.dtype, device="cuda")
        wide[:, :-1, off:off + d] = t
        return wide[:, :-1, off:off + d], wide

    def left(*wides):
        for wide in wides:
            assert (wide[:, -1] == 7.0).all() and (wide[..., :off] == 7.0).all() and (wide[..., off + d:] == 7.0).all()
    (q, wq), (k, wk) = part(x["q"]), part(x["k"])
    a, b = kda.qk_norm_rotary(q, k, q_out=q, k_out=k, **args)
    assert a is q and b is k
    ref.check("in place q", q, *want["q"])
    ref.check("in place k", k, *want["k"])
    left(wq, wk)
    (dq, wq), (dk, wk) = part(x["dq_out"]), part(x["dk_out"])
    got = kda.qk_norm_rotary_backward(x["q"], x["k"], dq, dk, dq=dq, dk=dk, **args)
    assert got["dq"] is dq and got["dk"] is dk
    for n in got:
        ref.check(f"onto dy {n}", got[n], *want[n])
    left(wq, wk)
    (q, wq), (k, wk) = part(x["q"]), part(x["k"])
    got = kda.qk_norm_rotary_backward(q, k, x["dq_out"], x["dk_out"], dq=q, dk=k, **args)
    for n in got:
        ref.check(f"onto x {n}", got[n], *want[n])
    left(wq, wk)
    grad = torch.full((T, H + 2 * Hk, d), 7.0, dtype=DT[dtype], device="cuda")
    got = kda.qk_norm_rotary_backward(x["q"], x["k"], x["dq_out"], x["dk_out"], dq=grad[:, :H], dk=grad[:, H:H + Hk], **args)
    for n in got:
        ref.check(f"parts of one gradient {n}", got[n], *want[n])
    assert (grad[:, H + Hk:] == 7.0).all()


def test_broadcast_inputs():
    """Strides of 0: one head, or one token, read by all."""
    import gated_delta_rule_prefill_amd as kda
    x = make(55, "bf16", 20, 4, 2, 64, 32)
    args = {n: x[n] for n in ("q_weight", "k_weight", "positions", "inv_freq")}
    one, tok = x["q"][:, :1].expand(-1, 4, -1), x["k"][:1].expand(20, -1, -1)
    got = kda.qk_norm_rotary(one, tok, **args)
    want = kda.qk_norm_rotary(one.contiguous(), tok.contiguous(), **args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a = kda.qk_norm_rotary_backward(one, tok, x["dq_out"], x["dk_out"], **args)
    b = kda.qk_norm_rotary_backward(one.contiguous(), tok.contiguous(), x["dq_out"], x["dk_out"], **args)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_rows_of_zeros_and_nothing_to_do():
    import gated_delta_rule_prefill_amd as kda
    x = make(56, "f32", 10, 2, 1, 64, 64)
    x["q"][3] = 0.0
    yq, _, g = check("zeros", x, eps=1e-5)
    assert (yq[3] == 0).all() and torch.isfinite(g["dq"]).all()
    x = make(57, "bf16", 0, 2, 1, 64, 64)
    args = {n: x[n] for n in ("q_weight", "k_weight", "positions", "inv_freq")}
    assert kda.qk_norm_rotary(x["q"], x["k"], **args)[0].shape == (0, 2, 64)
    g = kda.qk_norm_rotary_backward(x["q"], x["k"], x["dq_out"], x["dk_out"], **args)
    assert (g["dq_weight"] == 0).all() and (g["dk_weight"] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 80, 34])
def test_writes_stay_in_bounds(dtype, d):
    import gated_delta_rule_prefill_amd as kda
    T, H, Hk, t = 21, 3, 1, DT[dtype]
    x = make(58, dtype, T, H, Hk, d, 16)
    args = {n: x[n] for n in ("q_weight", "k_weight", "positions", "inv_freq")}
    need = kda.qk_norm_rotary_backward_workspace_bytes(d)
    out = dict(q_out=Guarded((T, H, d), t), k_out=Guarded((T, Hk, d), t), dq=Guarded((T, H, d), t), dk=Guarded((T, Hk, d), t),
               ws=Guarded((need,), torch.uint8, init=torch.full((need,), 255, dtype=torch.uint8, device="cuda")))
    kda.qk_norm_rotary(x["q"], x["k"], q_out=out["q_out"].t, k_out=out["k_out"].t, **args)
    g = kda.qk_norm_rotary_backward(x["q"], x["k"], x["dq_out"], x["dk_out"], dq=out["dq"].t, dk=out["dk"].t,
                                    workspace=out["ws"].t, **args)
    _check(out, f"norm {dtype} {d}")
    assert torch.isfinite(g["dq_weight"]).all()


def test_gradients_against_differences():
    """fp32, along random directions: step 2^-6 on unit directions; the fp32 error of
    the sum over 2h and h^2 times the third derivative stay under 2 % of the scale."""
    import gated_delta_rule_prefill_amd as kda
    x = make(59, "f32", 30, 3, 2, 64, 32)
    rot = dict(positions=x["positions"], inv_freq=x["inv_freq"], start=8, mscale=1.1)

    def f(**kw):
        y = {n: kw.get(n, x[n]) for n in ("q", "k", "q_weight", "k_weight")}
        a, b = kda.qk_norm_rotary(**y, **rot)
        return float((a.double() * x["dq_out"].double()).sum() + (b.double() * x["dk_out"].double()).sum())
    g = kda.qk_norm_rotary_backward(x["q"], x["k"], x["dq_out"], x["dk_out"], q_weight=x["q_weight"],
                                    k_weight=x["k_weight"], **rot)
    gen = torch.Generator().manual_seed(7)
    for name in ("q", "k", "q_weight", "k_weight"):
        grad = g["d" + name].double()
        direction = torch.randn(x[name].shape, generator=gen).cuda()
        for way in (direction / direction.norm(), (grad / grad.norm()).float()):
            h = 2.0 ** -6
            diff = (f(**{name: x[name] + h * way}) - f(**{name: x[name] - h * way})) / (2 * h)
            assert abs(diff - float((grad * way.double()).sum())) <= 0.02 * float(grad.norm()), name


def test_graph_and_streams():
    """Captured once, replayed on new inputs with eager calls in between; on
    another stream; deterministic, so bit for bit."""
    import gated_delta_rule_prefill_amd as kda
    xs = [make(60 + i, "bf16", 700, 4, 2, 128, 128) for i in range(3)]
    s = {n: t.clone() for n, t in xs[0].items()}

    def step(x, **kw):
        args = {n: x[n] for n in ("q_weight", "k_weight", "positions", "inv_freq")}
        return list(kda.qk_norm_rotary(x["q"], x["k"], **args, **kw)) + \
            list(kda.qk_norm_rotary_backward(x["q"], x["k"], x["dq_out"], x["dk_out"], **args, **kw).values())
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
        torch.cuda.synchronize()
        got = step(x, stream=side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
