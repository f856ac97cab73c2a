"""The window operators' entry points without a GPU: bad arguments are rejected
before any HIP call, with the status the header documents, and by the binding."""
import math

import pytest
import torch

from gated_delta_rule_prefill_amd import kda

A = 1 << 20  # a 16-byte-aligned fake device address; never dereferenced here
OK, INVALID, UNSUPPORTED, WORKSPACE = (kda.KDA_OK, kda.KDA_ERR_INVALID_ARGUMENT, kda.KDA_ERR_UNSUPPORTED,
                                       kda.KDA_ERR_WORKSPACE)
BF16 = kda.KDA_DTYPE_BF16


def _inputs(**kw):
    d = dict(q=A, k=A, v=A, qt=1024, qh=128, kt=512, kh=128, vt=512, vh=128, cu_q=A, cu_k=None, total_q=100, total_k=100,
             N=2, H=8, Hk=2, d=128, dtype=BF16, window=10, sinks=4, scale=0.1)   # in the order of kda_window_inputs
    d.update(kw)
    return kda._WINDOW.pack(*(x or 0 for x in d.values()))


BAD_INPUTS = [
    (dict(N=0), INVALID), (dict(H=0), INVALID), (dict(H=65536, Hk=8), INVALID), (dict(Hk=0), INVALID), (dict(Hk=3), INVALID),
    (dict(Hk=-2), INVALID), (dict(total_q=-1), INVALID), (dict(total_q=1 << 31, total_k=1 << 31), INVALID),
    (dict(total_q=1 << 30, total_k=1 << 30), INVALID), (dict(dtype=2), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED), (dict(window=0), INVALID), (dict(window=-5), INVALID), (dict(sinks=-1), INVALID),
    (dict(sinks=65), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(total_k=99), INVALID), (dict(cu_q=None, cu_k=A), INVALID),
    (dict(cu_q=None, N=3), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k=A + 8), INVALID), (dict(q=A + 2), INVALID), (dict(qt=7), INVALID), (dict(kh=-8), INVALID),
    (dict(vt=1 << 23), INVALID), (dict(kt=1 << 41), INVALID), (dict(N=300, total_q=300, total_k=300, H=65408, Hk=65408), INVALID),
    (dict(N=1 << 23), INVALID), (dict(total_q=1 << 28, total_k=1 << 28, H=64, Hk=8), INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_INPUTS)
def test_attention_rejects(kw, status):
    a = _inputs(**kw)
    assert kda.lib().kda_window_attention(a, A, A, None) == status and kda.last_error()
    assert _backward(inputs=kw) == status and kda.last_error()


def test_attention_rejects_outputs_and_accepts_nothing_to_do():
    lib, a = kda.lib(), _inputs()
    assert lib.kda_window_attention(None, A, A, None) == INVALID
    assert lib.kda_window_attention(a, None, A, None) == INVALID
    assert lib.kda_window_attention(a, A, A + 4, None) == INVALID
    a = _inputs(total_q=0, total_k=0)
    assert lib.kda_window_attention(a, None, None, None) == OK
    assert _backward(inputs=dict(total_q=0, total_k=0), o=None, lse=None, d_o=None, dq=None, dk=None, dv=None) == OK


def _backward(inputs=None, **kw):
    d = dict(o=A, lse=A, d_o=A, dq=A, dk=A, dkt=512, dkh=128, dv=A, dvt=512, dvh=128, ws=A, wsb=1 << 40)
    d.update(kw)
    return kda.lib().kda_window_attention_backward(_inputs(**(inputs or {})), *d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(d_o=None), INVALID), (dict(dq=None), INVALID),
    (dict(dk=None), INVALID), (dict(dv=None), INVALID), (dict(dv=A + 2), INVALID), (dict(dkt=3), INVALID),
    (dict(dkh=64), INVALID), (dict(dvt=0), INVALID), (dict(ws=None), INVALID), (dict(ws=A + 8), INVALID),
    (dict(wsb=100), WORKSPACE), (dict(inputs=dict(N=1 << 23, H=1, Hk=1)), INVALID),
])
def test_backward_rejects(kw, status):
    assert _backward(**kw) == status and kda.last_error()


def test_backward_workspace():
    """Never falls as an argument grows; 0 for sizes that a call refuses."""
    w = kda.window_attention_backward_workspace_bytes
    last = 0
    for T in (0, 1, 1000, 1024, 5000, 100000):
        now = w(T, 4, 8, 2, 128, 4)
        assert now >= last and now % 256 == 0
        last = now
    assert w(1000, 4, 8, 2, 128, 4) <= w(1000, 5, 8, 2, 128, 4) <= w(1000, 5, 8, 4, 128, 4) <= w(1000, 5, 8, 4, 128, 64)
    assert w(1000, 4, 8, 2, 64, 4) <= w(1000, 4, 8, 2, 128, 4)
    for bad in ((-1, 4, 8, 2, 128, 4), (1000, 0, 8, 2, 128, 4), (1000, 4, 8, 3, 128, 4), (1000, 4, 8, 2, 96, 4),
                (1000, 4, 8, 2, 128, 65), (1000, 4, 0, 2, 128, 4)):
        assert w(*bad) == 0
    assert kda.window_decode_workspace_bytes(96) == 0 and kda.window_decode_workspace_bytes(128) > 0
    assert kda.qk_norm_rotary_backward_workspace_bytes(258) == 0 and kda.qk_norm_rotary_backward_workspace_bytes(6) > 0


def _cache(**kw):
    d = dict(k=A, v=A, ps=16 * 256, ts=256, hs=128, table=A, lens=A, P=10, page=16, maxp=4)   # in kda_kv_cache's order
    d.update(kw)
    return kda._KV_CACHE.pack(*(x or 0 for x in d.values()))


def _decode(cache=None, **kw):
    d = dict(q=A, qt=1024, qh=128, cu=A, T=2, N=2, H=8, Hk=2, d=128, dtype=BF16, window=10, sinks=4, scale=0.1, o=A, lse=A,
             ws=A, wsb=1 << 40)
    d.update(kw)
    return kda.lib().kda_window_decode(_cache(**(cache or {})), *d.values(), None)


def _append(cache=None, **kw):
    d = dict(k=A, kt=512, kh=128, v=A, vt=512, vh=128, cu=A, T=2, N=2, Hk=2, d=128, dtype=BF16, w=A, eps=1e-6, f=A, start=0,
             dr=64, amp=1.0, flags=0, out=A)
    d.update(kw)
    return kda.lib().kda_kv_append(_cache(**(cache or {})), *d.values(), None)


BAD_CACHES = [dict(P=0), dict(page=0), dict(maxp=0), dict(P=1 << 30, page=4), dict(maxp=1 << 30, page=4), dict(k=None),
              dict(v=None), dict(table=None), dict(lens=None), dict(k=A + 8), dict(v=A + 4), dict(ps=3), dict(ts=-256),
              dict(hs=1 << 41)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_caches_rejected(kw):
    assert _decode(cache=kw) == INVALID and kda.last_error()
    assert _append(cache=kw) == INVALID and kda.last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), INVALID), (dict(N=0), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID),
    (dict(cu=None, T=3), INVALID), (dict(H=0), INVALID), (dict(H=7), INVALID), (dict(Hk=0), INVALID),
    (dict(d=32), UNSUPPORTED), (dict(window=0), INVALID), (dict(sinks=65), INVALID), (dict(scale=math.nan), INVALID),
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(q=A + 8), INVALID), (dict(lse=A + 4), INVALID),
    (dict(qt=4), INVALID), (dict(qh=-128), INVALID), (dict(ws=None), INVALID), (dict(wsb=16), WORKSPACE),
    (dict(T=1 << 29, H=8, Hk=8), INVALID), (dict(N=1 << 23, T=0), INVALID),
])
def test_decode_rejects(kw, status):
    assert _decode(**kw) == status and kda.last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), INVALID), (dict(N=0), INVALID), (dict(T=-1), INVALID), (dict(cu=None, T=3), INVALID),
    (dict(Hk=0), INVALID), (dict(d=256), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k=A + 8), INVALID), (dict(out=A + 8), INVALID), (dict(w=A + 4), INVALID), (dict(kt=4), INVALID),
    (dict(vh=-8), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(amp=math.inf), INVALID),
    (dict(start=-2), INVALID), (dict(start=66), INVALID), (dict(dr=130), INVALID), (dict(dr=3), INVALID),
    (dict(dr=-2), INVALID), (dict(dr=0), INVALID), (dict(f=None), INVALID), (dict(flags=2), INVALID),
    (dict(cache=dict(hs=64)), INVALID), (dict(cache=dict(ts=64)), INVALID), (dict(cache=dict(ps=0)), INVALID),
])
def test_append_rejects(kw, status):
    assert _append(**kw) == status and kda.last_error()


def test_no_tokens():
    assert _decode(T=0, q=None, o=None, lse=None) == OK
    assert _append(T=0, k=None, v=None, out=None) == OK
    assert kda.lib().kda_window_decode(None, A, 1024, 128, A, 2, 2, 8, 2, 128, BF16, 10, 4, 0.1, A, A, A, 1 << 40,
                                       None) == INVALID
    assert kda.lib().kda_kv_append(None, A, 512, 128, A, 512, 128, A, 2, 2, 2, 128, BF16, A, 1e-6, A, 0, 64, 1.0, 0, A,
                                   None) == INVALID


def _heads(**kw):
    d = dict(x=A, xt=512, xh=128, y=2 * A, yt=512, yh=128, w=A, dy=3 * A, dyt=512, dyh=128, dx=4 * A, dxt=512, dxh=128, dw=A,
             H=4)   # in kda_norm_heads' order
    d.update(kw)
    return kda._NORM_HEADS.pack(*(x or 0 for x in d.values()))


def _norm(backward, q=None, k=None, heads=True, **kw):
    d = dict(pos=A, f=A, T=10, d=128, start=0, dr=64, dtype=BF16, eps=1e-6, amp=1.0, flags=0)
    ws = {n: kw.pop(n) for n in ("ws", "wsb") if n in kw}
    d.update(kw)
    a, b = _heads(**(q or {})) if heads else None, None if k is None else _heads(**k)
    if backward:
        return kda.lib().kda_qk_norm_rotary_backward(a, b, *d.values(), ws.get("ws", A), ws.get("wsb", 1 << 40), None)
    return kda.lib().kda_qk_norm_rotary(a, b, *d.values(), None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(heads=False), INVALID), (dict(dtype=3), INVALID), (dict(flags=2), INVALID), (dict(T=-1), INVALID),
    (dict(T=1 << 31), INVALID), (dict(d=0), UNSUPPORTED), (dict(d=63), UNSUPPORTED), (dict(d=258), UNSUPPORTED),
    (dict(dr=-2), INVALID), (dict(dr=7), INVALID), (dict(start=-1), INVALID), (dict(start=70), INVALID),
    (dict(dr=130), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=math.inf), INVALID), (dict(amp=math.nan), INVALID),
    (dict(dr=0), INVALID), (dict(pos=None), INVALID), (dict(f=None), INVALID), (dict(pos=A + 4), INVALID),
    (dict(q=dict(H=0)), INVALID), (dict(k=dict(H=70000)), INVALID), (dict(k=dict(x=None)), INVALID),
    (dict(q=dict(x=A + 1)), INVALID), (dict(q=dict(w=A + 4)), INVALID), (dict(q=dict(xt=-1)), INVALID),
    (dict(k=dict(xh=1 << 40)), INVALID),
])
def test_norm_rejects(backward, kw, status):
    assert _norm(backward, **kw) == status and kda.last_error()


@pytest.mark.parametrize("backward,kw,status", [
    (False, dict(q=dict(y=None)), INVALID), (False, dict(q=dict(y=A + 1)), INVALID), (False, dict(q=dict(yh=64)), INVALID),
    (False, dict(k=dict(yt=100)), INVALID), (False, dict(q=dict(y=A, yt=1024)), INVALID),
    (True, dict(q=dict(dy=None)), INVALID), (True, dict(k=dict(dx=None)), INVALID), (True, dict(q=dict(dxh=64)), INVALID),
    (True, dict(q=dict(dw=A + 8)), INVALID), (True, dict(q=dict(dx=A, dxt=1024)), INVALID),
    (True, dict(q=dict(dx=3 * A, dxh=256)), INVALID), (True, dict(k=dict(dyt=-1)), INVALID),
    (True, dict(ws=None), INVALID), (True, dict(wsb=64), WORKSPACE), (True, dict(ws=A + 8), INVALID),
])
def test_norm_rejects_outputs(backward, kw, status):
    assert _norm(backward, **kw) == status and kda.last_error()


def test_norm_without_tokens():
    none = dict(x=None, y=None, dy=None, dx=None, dw=None)
    assert _norm(False, q=none, k=none, T=0, pos=None, f=None) == OK
    assert _norm(True, q=none, k=none, T=0, pos=None, f=None) == OK


# -- the binding ---------------------------------------------------------------------

def _t(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


@pytest.mark.parametrize("kw", [
    dict(q=_t(10, 8, 64)), dict(q=_t(10, 8)), dict(v=_t(10, 2, 64)), dict(v=_t(9, 2, 128)),
    dict(k=_t(10, 2, 128, dtype=torch.float32)), dict(q=_t(10, 8, 256)[..., ::2]), dict(cu_seqlens_k=_t(3, dtype=torch.int32)),
    dict(cu_seqlens=_t(3, dtype=torch.int64)), dict(window=1 << 31), dict(num_seqs=1 << 31), dict(),
])
def test_attention_binding_rejects(kw):
    """CPU tensors with everything else in order are refused as well (the last)."""
    a = dict(q=_t(10, 8, 128), k=_t(10, 2, 128), v=_t(10, 2, 128), window=4)
    a.update(kw)
    with pytest.raises(ValueError):
        kda.window_attention(**a)
    with pytest.raises(ValueError):
        kda.window_attention_backward(o=_t(10, 8, 128), lse=_t(10, 8, dtype=torch.float32), d_o=_t(10, 8, 128), **a)


_I = torch.int32


@pytest.mark.parametrize("kw", [
    dict(k_cache=_t(4, 16, 2)), dict(v_cache=_t(4, 16, 2, 64)), dict(v_cache=_t(4, 2, 16, 128).transpose(1, 2)),
    dict(v_cache=_t(4, 16, 2, 128, dtype=torch.float32)), dict(block_table=_t(3, 4, dtype=_I)),
    dict(block_table=_t(2, 4, dtype=torch.int64)), dict(seq_lens=_t(3, dtype=_I)), dict(seq_lens=_t(2, dtype=torch.int64)),
    dict(cu_seqlens=_t(4, dtype=_I)), dict(k_cache=_t(4, 16, 2, 256)[..., ::2], v_cache=_t(4, 16, 2, 256)[..., ::2]), dict(),
])
def test_cache_binding_rejects(kw):
    a = dict(k_cache=_t(4, 16, 2, 128), v_cache=_t(4, 16, 2, 128), block_table=_t(2, 4, dtype=_I), seq_lens=_t(2, dtype=_I))
    a.update(kw)
    with pytest.raises(ValueError):
        kda.window_decode(_t(2, 8, 128), window=4, **a)
    with pytest.raises(ValueError):
        kda.kv_append(k=_t(2, 2, 128), v=_t(2, 2, 128), **a)


@pytest.mark.parametrize("kw", [
    dict(q=_t(10, 512)), dict(k=_t(9, 2, 128)), dict(k=_t(10, 2, 64)), dict(q_weight=_t(64, dtype=torch.float32)),
    dict(q_weight=_t(128)), dict(k=None), dict(positions=None), dict(inv_freq=None), dict(positions=_t(9, dtype=_I)),
    dict(positions=_t(10, dtype=torch.int64)), dict(),
])
def test_norm_binding_rejects(kw):
    a = dict(q=_t(10, 4, 128), k=_t(10, 2, 128), k_weight=_t(128, dtype=torch.float32), positions=_t(10, dtype=_I),
             inv_freq=_t(32, dtype=torch.float32))
    a.update(kw)
    with pytest.raises(ValueError):
        kda.qk_norm_rotary(**a)
    with pytest.raises(ValueError):
        kda.qk_norm_rotary_backward(dq_out=_t(10, 4, 128), dk_out=_t(10, 2, 128), **a)
