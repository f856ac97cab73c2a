"""The window operators' host side over a stand-in for HIP (hip_stub.py): what is
launched, and what happens when a launch is refused."""
import pytest

import hip_stub
from gated_delta_rule_prefill_amd import kda

SETUP = """
def window(cu_q=None, cu_k=None, bf16=True, T=300, window=64, sinks=4):
    return kda._WINDOW.pack(A, A, A, 1024, 128, 512, 128, 512, 128, address(cu_q), address(cu_k), T, T, 2, 8, 2, 128,
                            1 if bf16 else 0, window, sinks, 0.1)

def w_forward(**kw):
    return lib.kda_window_attention(window(**kw), A, A, None)

def w_backward(ws=A, **kw):
    return lib.kda_window_attention_backward(window(**kw), A, A, A, A, A, 512, 128, A, 512, 128, ws,
                                             (1 << 40) if ws else 0, None)

kv = kda._KV_CACHE.pack(A, A, 16 * 256, 256, 128, A, A, 1000, 16, 300)

def w_decode(cu=None, T=2, bf16=True, ws=A, window=4096, N=2):
    return lib.kda_window_decode(kv, A, 1024, 128, address(cu), T, N, 8, 2, 128, int(bf16), window, 4, 0.1, A, A, ws,
                                 (1 << 40) if ws else 0, None)

def w_append(cu=None):
    return lib.kda_kv_append(kv, A, 512, 128, A, 512, 128, address(cu), 2, 2, 2, 128, 1, A, 1e-6, A, 0, 64, 1.0, 0, A, None)

def heads(n):
    return kda._NORM_HEADS.pack(n * A, 512, 128, (n + 1) * A, 512, 128, A, (n + 2) * A, 512, 128, (n + 3) * A, 512, 128, A, 4)

def w_norm(dtype=1, T=10):
    return lib.kda_qk_norm_rotary(heads(1), heads(9), A, A, T, 128, 0, 64, dtype, 1e-6, 1.0, 0, None)

def w_norm_backward(dtype=1, T=10, ws=A):
    return lib.kda_qk_norm_rotary_backward(heads(1), heads(9), A, A, T, 128, 0, 64, dtype, 1e-6, 1.0, 0, ws,
                                           (1 << 40) if ws else 0, None)
"""

CALLS = {   # call -> its launches
    "forward": ("w_forward", 1), "backward": ("w_backward", 3), "backward without sinks": ("w_backward, sinks=0", 2),
    "backward with a window over all": ("w_backward, window=300", 2), "backward in fp32": ("w_backward, bf16=False", 3),
    "backward without a workspace": ("w_backward, ws=None", 3),
    "decode, split": ("w_decode", 2), "decode, short window": ("w_decode, window=64", 1),
    "decode, many sequences": ("w_decode, T=600, N=600", 1), "decode, many rows": ("w_decode, T=3000", 1), "decode, a few rows": ("w_decode, T=60", 2),
    "decode without a workspace": ("w_decode, ws=None", 2), "append": ("w_append", 1), "norm": ("w_norm", 1),
    "norm backward": ("w_norm_backward", 2), "norm backward without tokens": ("w_norm_backward, T=0", 1),
    "norm backward without a workspace": ("w_norm_backward, ws=None", 2),
}


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    code = SETUP + "".join(f"result[{name!r}] = [call({f.split(',')[0]}, r{','.join([''] + f.split(',')[1:])}) "
                           f"for r in range({n + 1})]\n" for name, (f, n) in CALLS.items())
    return hip_stub.run(tmp_path_factory.mktemp("stub"), code)


@pytest.mark.parametrize("name", CALLS)
def test_a_refused_launch_ends_the_call(calls, name):
    """Nothing is launched behind a refused launch: the next kernel would read
    what the refused one did not write."""
    plain, *refused = calls[name]
    n = CALLS[name][1]
    assert plain == dict(status=kda.KDA_OK, launches=n, syncs=0, text="")
    for at, got in enumerate(refused, 1):
        assert (got["status"], got["launches"]) == (kda.KDA_ERR_HIP, at) and "refused" in got["text"]


def test_debug_sync(tmp_path):
    """With KDA_DEBUG_SYNC=1 the operators wait for the stream behind every kernel,
    and refuse offsets that decrease before they launch any."""
    code = SETUP + "".join(f"result[{name!r}] = call({f.split(',')[0]}{','.join([''] + f.split(',')[1:])})\n"
                           for name, (f, n) in CALLS.items())
    code += """
down, rising = offsets(0, 200, 150), offsets(5, 200, 290)
for name, f, kw in (("q", w_forward, "cu_q"), ("k", w_forward, "cu_k"), ("dq", w_backward, "cu_q"),
                    ("dk", w_backward, "cu_k"), ("decode", w_decode, "cu"), ("append", w_append, "cu")):
    result["offsets " + name] = [call(f, **dict({"cu_q": rising} if kw == "cu_k" else {}, **{kw: cu}))
                                 for cu in (down, rising)]
"""
    got = hip_stub.run(tmp_path, code, KDA_DEBUG_SYNC="1")
    for name, (_, n) in CALLS.items():
        assert got[name] == dict(status=kda.KDA_OK, launches=n, syncs=n, text=""), name
    for name in ("q", "k", "dq", "dk", "decode", "append"):
        down, rising = got["offsets " + name]
        assert down["status"] == kda.KDA_ERR_INVALID_ARGUMENT and "non-decreasing" in down["text"], name
        assert down["launches"] == 0
        copies = 2 if name in ("k", "dk") else 1
        assert rising["status"] == kda.KDA_OK and rising["syncs"] == rising["launches"] + copies, name
