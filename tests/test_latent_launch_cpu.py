"""The latent operators' host side over a stand-in for HIP (hip_stub.py): what
is launched, and what happens when a launch is refused."""
import pytest

import hip_stub
from gated_delta_rule_prefill_amd import kda

CALLS = {   # call -> its launches
    "decode": ("decode", 2), "decode many rows": ("decode, T=200, H=32", 2), "decode fp32": ("decode, bf16=False", 2),
    "decode without a workspace": ("decode, ws=None", 2), "append": ("append", 1), "rotary": ("rotary", 1),
    "forward": ("forward", 1), "backward": ("backward", 3), "backward without key parts": ("backward, dr=0", 2),
    "backward in fp32, split": ("backward, bf16=False", 3), "backward in fp32, whole": ("backward, bf16=False, T=9000", 3),
}


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    code = "".join(f"result[{name!r}] = [call({f.split(',')[0]}, r{','.join([''] + f.split(',')[1:])}) "
                   f"for r in range({n + 1})]\n" for name, (f, n) in CALLS.items())
    return hip_stub.run(tmp_path_factory.mktemp("stub"), code)


@pytest.mark.parametrize("name", CALLS)
def test_a_refused_launch_ends_the_call(calls, name):
    """Nothing is launched behind a refused launch: the next kernel would read
    what the refused one did not write (a join follows row numbers that the
    decode kernel leaves in the workspace)."""
    plain, *refused = calls[name]
    n = CALLS[name][1]
    assert plain == dict(status=kda.KDA_OK, launches=n, syncs=0, text="")
    for at, got in enumerate(refused, 1):
        assert (got["status"], got["launches"]) == (kda.KDA_ERR_HIP, at) and "refused" in got["text"]


def test_debug_sync(tmp_path):
    """With KDA_DEBUG_SYNC=1 the latent operators wait for the stream behind every
    kernel, and refuse offsets that decrease before they launch any."""
    code = "".join(f"result[{name!r}] = call({f.split(',')[0]}{','.join([''] + f.split(',')[1:])})\n"
                   for name, (f, n) in CALLS.items())
    code += """
down, rising = offsets(0, 200, 150), offsets(5, 200, 290)
for name, f, kw in (("q", forward, "cu_q"), ("k", forward, "cu_k"), ("dq", backward, "cu_q"), ("dk", backward, "cu_k"),
                    ("decode", decode, "cu"), ("append", append, "cu")):
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


def test_rotary_in_place_with_strides_of_axes_of_one(tmp_path):
    """The stride of one token, or of one head, is not looked at."""
    code = """
def turn(T, H, xt, xh):
    return lib.kda_rotary(A, xt, xh, A, 256, 64, A, A, T, H, 64, 0, 64, 1, 1.0, 0, None)
result["token"], result["head"] = call(turn, T=1, H=4, xt=0, xh=64), call(turn, T=3, H=1, xt=256, xh=0)
"""
    for got in hip_stub.run(tmp_path, code).values():
        assert got["status"] == kda.KDA_OK and got["launches"] == 1
