"""The latent-attention entry points without a GPU: bad arguments are rejected
before any HIP call, with the status the header documents."""
import math

import pytest

from gated_delta_rule_prefill_amd import kda

A = 1 << 20  # a 16-byte-aligned fake device address; never dereferenced here
INVALID, UNSUPPORTED, WORKSPACE = (kda.KDA_ERR_INVALID_ARGUMENT, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE)


def _inputs(**kw):
    d = dict(q=A, k=A, v=A, k_pe=A, q_token_stride=768, q_head_stride=192, k_token_stride=1024, k_head_stride=256,
             v_token_stride=1024, v_head_stride=256, k_pe_token_stride=64, cu_seqlens_q=A, cu_seqlens_k=None,
             total_q=100, total_k=100, num_seqs=2, H=4, dn=128, dr=64, dv=128, dtype=kda.KDA_DTYPE_BF16, causal=1,
             scale=0.1)   # in the order of kda_latent_inputs
    d.update(kw)
    return kda._INPUTS.pack(*(x or 0 for x in d.values()))


BAD_INPUTS = [
    (dict(num_seqs=0), INVALID), (dict(H=0), INVALID), (dict(H=70000), INVALID), (dict(total_q=-1), INVALID),
    (dict(total_q=1 << 31, total_k=1 << 31), INVALID), (dict(dtype=2), INVALID), (dict(dn=96, dv=96), UNSUPPORTED),
    (dict(dv=64), UNSUPPORTED), (dict(dr=32), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(total_k=99), INVALID), (dict(cu_seqlens_q=None, cu_seqlens_k=A), INVALID),
    (dict(cu_seqlens_q=None, num_seqs=3), INVALID), (dict(q=None), INVALID), (dict(v=None), INVALID),
    (dict(k_pe=None), INVALID), (dict(k=A + 8), INVALID), (dict(q_token_stride=7), INVALID),
    (dict(k_head_stride=-8), INVALID), (dict(total_q=2 ** 30, total_k=2 ** 30, H=65535), INVALID), (dict(k_token_stride=1 << 23), INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_INPUTS)
def test_attention_rejects(kw, status):
    a = _inputs(**kw)
    assert kda.lib().kda_latent_attention(a, A, A, None) == status
    assert kda.last_error()


def test_attention_rejects_outputs_and_accepts_nothing_to_do():
    lib, a = kda.lib(), _inputs()
    assert lib.kda_latent_attention(None, A, A, None) == INVALID
    assert lib.kda_latent_attention(a, None, A, None) == INVALID
    assert lib.kda_latent_attention(a, A + 4, A, None) == INVALID
    a = _inputs(total_q=0, total_k=0)
    assert lib.kda_latent_attention(a, None, None, None) == kda.KDA_OK


def _backward(inputs=None, **kw):
    d = dict(o=A, lse=A, d_o=A, dq=A, dk=A, dkt=1024, dkh=256, dv=A, dvt=1024, dvh=256, pe=A, ws=A, wsb=1 << 40)
    d.update(kw)
    a = _inputs(**(inputs or {}))
    return kda.lib().kda_latent_attention_backward(a, d["o"], d["lse"], d["d_o"], d["dq"], d["dk"],
                                                   d["dkt"], d["dkh"], d["dv"], d["dvt"], d["dvh"], d["pe"], d["ws"],
                                                   d["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID),
    (dict(pe=None), INVALID), (dict(dv=A + 2), INVALID), (dict(dkt=3), INVALID), (dict(dkh=64), INVALID),
    (dict(dvt=0), INVALID), (dict(ws=None), INVALID), (dict(wsb=100), WORKSPACE),
    (dict(inputs=dict(dn=32)), UNSUPPORTED),
])
def test_backward_rejects(kw, status):
    assert _backward(**kw) == status
    assert kda.last_error()


def _decode(**kw):
    d = dict(q=A, qt=576 * 4, qh=576, cache=A, P=10, page=64, table=A, maxp=4, lens=A, cu=A, T=2, N=2, H=4, dl=512,
             dr=64, dtype=kda.KDA_DTYPE_BF16, scale=0.1, o=A, lse=A, ws=A, wsb=1 << 40)
    d.update(kw)
    return kda.lib().kda_latent_decode(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), INVALID), (dict(N=0), INVALID), (dict(T=-1), INVALID), (dict(P=0), INVALID),
    (dict(page=0), INVALID), (dict(maxp=0), INVALID), (dict(P=1 << 30, page=4), INVALID),
    (dict(maxp=1 << 30, page=4), INVALID), (dict(cu=None, T=3), INVALID), (dict(cache=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(H=0), INVALID), (dict(dl=128), UNSUPPORTED),
    (dict(dr=32), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(q=None), INVALID),
    (dict(o=A + 8), INVALID), (dict(qt=4), INVALID), (dict(ws=None), INVALID), (dict(wsb=64), WORKSPACE),
])
def test_decode_rejects(kw, status):
    assert _decode(**kw) == status
    assert kda.last_error()


def test_decode_nothing_to_do():
    assert _decode(T=0, q=None, o=None) == kda.KDA_OK


def _append(**kw):
    d = dict(cache=A, P=10, page=64, table=A, maxp=4, lens=A, cu=A, T=2, N=2, dl=512, dr=64,
             dtype=kda.KDA_DTYPE_BF16, c=A, ct=576, pe=A, pet=576, w=A, eps=1e-6, f=A, amp=1.0, flags=0, co=A, po=A)
    d.update(kw)
    return kda.lib().kda_latent_append(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), INVALID), (dict(flags=2), INVALID), (dict(flags=4), INVALID), (dict(N=0), INVALID),
    (dict(page=-1), INVALID), (dict(dl=500), UNSUPPORTED), (dict(dl=2048), UNSUPPORTED), (dict(dr=4), UNSUPPORTED),
    (dict(dr=512), UNSUPPORTED), (dict(c=None), INVALID), (dict(pe=None), INVALID),
    (dict(dr=0, f=None), INVALID), (dict(dr=0, po=None), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=math.nan), INVALID), (dict(amp=math.inf), INVALID), (dict(ct=5), INVALID), (dict(co=A + 2), INVALID),
    (dict(cu=None, T=3), INVALID),
])
def test_append_rejects(kw, status):
    assert _append(**kw) == status
    assert kda.last_error()


def _rotary(**kw):
    d = dict(x=A, xt=256, xh=64, y=2 * A, yt=256, yh=64, pos=A, f=A, T=10, H=4, d=64, start=0, dr=64,
             dtype=kda.KDA_DTYPE_BF16, amp=1.0, flags=0)
    d.update(kw)
    return kda.lib().kda_rotary(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), INVALID), (dict(flags=4), INVALID), (dict(H=0), INVALID), (dict(T=-1), INVALID),
    (dict(d=5000), UNSUPPORTED), (dict(dr=3), INVALID), (dict(dr=0), INVALID), (dict(start=2), INVALID),
    (dict(start=-2), INVALID), (dict(start=2 ** 31 - 2), INVALID), (dict(amp=math.nan), INVALID),
    (dict(x=None), INVALID), (dict(pos=None), INVALID), (dict(x=A + 1), INVALID), (dict(xt=-1), INVALID),
    (dict(yh=32), INVALID), (dict(yt=0), INVALID), (dict(y=A, xt=512), INVALID),
])
def test_rotary_rejects(kw, status):
    assert _rotary(**kw) == status
    assert kda.last_error()


def test_workspace_sizes():
    lib = kda.lib()
    w = lib.kda_latent_attention_backward_workspace_bytes(4096, 4096, 32, 64)
    assert w >= 4096 * 32 * 4 + 4096 * 32 * 64 * 4 and w % 256 == 0
    assert lib.kda_latent_attention_backward_workspace_bytes(-1, 0, 32, 64) == 0
    assert lib.kda_latent_attention_backward_workspace_bytes(1, 1, 32, 60) == 0
    w = kda.latent_decode_workspace_bytes(256, 256, 32, 512, 64, True)
    assert w > 0 and w % 256 == 0
    assert kda.latent_decode_workspace_bytes(256, 0, 32, 512, 64, True) == 0
    assert kda.latent_decode_workspace_bytes(256, 256, 32, 100, 64, True) == 0


def test_rotary_frequencies():
    f, a = kda.rotary_frequencies(64)
    assert a == 1.0 and f.tolist() == [pytest.approx(10000.0 ** (-2 * i / 64), rel=2 ** -23) for i in range(32)]
    f, a = kda.rotary_frequencies(64, factor=4.0)
    assert a == 1.0 and f.tolist() == [pytest.approx(10000.0 ** (-2 * i / 64) / 4, rel=2 ** -23) for i in range(32)]
    f, a = kda.rotary_frequencies(64, factor=32.0, original_context=4096)
    assert a == pytest.approx(0.1 * math.log(32.0) + 1.0, rel=2 ** -23)
    for i, x in enumerate(f.tolist()):
        g = 10000.0 ** (-2 * i / 64)
        turns = 4096 * g / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 31))
        assert x == pytest.approx(g * keep + g / 32 * (1 - keep), rel=2 ** -22)
    for kw in (dict(dr=3), dict(dr=0), dict(dr=64, base=1.0), dict(dr=64, factor=0.5), dict(dr=64, factor=math.nan),
               dict(dr=64, original_context=-1)):
        with pytest.raises(kda.KDAError):
            kda.rotary_frequencies(**kw)


def test_binding_rejects_shapes_before_the_library():
    """Host tensors are enough for the binding's own checks."""
    import torch
    q, k = torch.zeros(4, 2, 192, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    pe = torch.zeros(4, 64, dtype=torch.bfloat16)
    ok = dict(k_pe=pe)
    for bad in (dict(k_pe=None), dict(k_pe=pe[:3]), dict(k_pe=pe.float()),
                dict(cu_seqlens=torch.zeros(3)), dict(cu_seqlens_k=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            kda.latent_attention(q, k, k, **{**ok, **bad})
    with pytest.raises(ValueError):
        kda.latent_attention(q, k.transpose(1, 2).contiguous().transpose(1, 2), k, **ok)
    cache, table = torch.zeros(3, 16, 320), torch.zeros(2, 1, dtype=torch.int32)
    lens = torch.ones(2, dtype=torch.int32)
    qd = torch.zeros(2, 4, 320)
    for bad in (dict(q=qd[..., :319]), dict(block_table=table.long()), dict(seq_lens=lens[:1]),
                dict(cache=cache.transpose(0, 1)), dict(cu_seqlens=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            kda.latent_decode(**{**dict(q=qd, cache=cache, block_table=table, seq_lens=lens, latent_dim=256, scale=1.0),
                                 **bad})
    with pytest.raises(ValueError):
        kda.latent_append(cache, torch.zeros(2, 256), table, lens)          # k_pe is missing
    with pytest.raises(ValueError):
        kda.rotary(torch.zeros(2, 1, 64), torch.zeros(2, dtype=torch.int64), torch.zeros(32))


def test_attention_rejects_more_tiles_than_a_grid_has():
    for kw in (dict(total_q=2 ** 28, total_k=2 ** 28, H=4, num_seqs=1), dict(num_seqs=2 ** 22, H=4)):
        a = _inputs(**kw)
        assert kda.lib().kda_latent_attention(a, A, A, None) == INVALID
        assert "too many tiles" in kda.last_error()


def test_workspace_of_a_large_batch_serves_smaller_ones():
    """The sizes never fall as an argument grows, though small batches are split
    over more workgroups and long rows take larger tiles."""
    import itertools
    lib = kda.lib()
    rows, heads = [0, 1, 63, 64, 65, 495, 1024, 2040, 2048, 4096, 30000], [1, 3, 4, 32, 128]
    for dr in (0, 64):
        size = {(q, k, h): lib.kda_latent_attention_backward_workspace_bytes(q, k, h, dr)
                for q, k, h in itertools.product(rows, rows, heads)}
        for (q, k, h), n in size.items():
            for bigger in ((rows[min(rows.index(q) + 1, 10)], k, h), (q, rows[min(rows.index(k) + 1, 10)], h),
                           (q, k, heads[min(heads.index(h) + 1, 4)])):
                assert size[bigger] >= n, (dr, (q, k, h), bigger)
    for dl, bf16 in itertools.product((256, 512), (True, False)):
        size = [kda.latent_decode_workspace_bytes(t, n, h, dl, 64, bf16)
                for t, n, h in ((1, 1, 1), (64, 64, 32), (64, 16, 32), (256, 256, 32), (257, 256, 32), (4096, 16, 128))]
        assert size == sorted(size) and size[0] > 0


def test_backward_bf16_needs_no_room_for_splits():
    """bf16 calls are never split: they ask for their row statistics and the heads'
    parts of dk_pe only."""
    rows = 100 * 4
    need = -(-rows * 8 // 256) * 256 + -(-rows * 64 * 4 // 256) * 256 + 256
    assert _backward(wsb=need - 1) == WORKSPACE
    assert "need %d bytes" % need in kda.last_error()
    assert _backward(inputs=dict(dtype=kda.KDA_DTYPE_F32), wsb=need) == WORKSPACE


def test_stream_of_another_device_is_refused():
    """Such a stream was dropped: the call ran on its tensors' device's current one."""
    from types import SimpleNamespace

    import torch
    there = SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        kda._elsewhere(torch.device("cuda", 0), there)


def test_no_sequences_are_refused():
    """num_seqs=0 is passed on, for the library to refuse, and not taken for 1."""
    import torch
    q, k = torch.zeros(4, 2, 64), torch.zeros(4, 2, 64)
    for num_seqs, n in ((None, 1), (2, 2), (0, 0), (-1, -1)):
        packed, _ = kda._latent_inputs(q, k, k, None, None, None, num_seqs, True, None)
        assert kda._INPUTS.unpack(packed)[15] == n
        if n < 1:
            assert kda.lib().kda_latent_attention(packed, A, A, None) == INVALID and "num_seqs" in kda.last_error()


def test_decode_rejects_more_rows_than_it_counts():
    for kw in (dict(T=1 << 26, N=1, H=32), dict(T=1 << 20, N=1 << 20, H=4096), dict(T=32769, N=32769, H=65535)):
        assert _decode(**kw) == INVALID
        assert "total_tokens * H" in kda.last_error()
    # the largest that is counted goes on to the next check
    assert _decode(T=(1 << 31) - 4096, N=1, H=1, q=None) == INVALID and "q and o" in kda.last_error()


def test_rotary_of_no_tokens():
    """Two empty tensors may have one address (NULL) and different strides."""
    for at in (None, A):
        assert _rotary(T=0, x=at, y=at, xt=320 * 4, xh=320, pos=None) == kda.KDA_OK
    # in place, strides of axes of one do not matter; those of others do
    assert _rotary(T=1, x=A, y=A, xh=128) == INVALID and "in place" in kda.last_error()
    assert _rotary(T=2, H=1, x=A, y=A, xt=512) == INVALID and "in place" in kda.last_error()
