"""Scores of -Inf: they weigh nothing, and a row all of whose scores are -Inf is as one
that sees no key (include/kda.h); its gradients are not finite."""
import pytest
import torch

import test_gpu_window_attention as ta
import test_gpu_window_decode as td

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("empty", [0, 600], ids=["split", "whole"])
def test_packed(dtype, empty):
    """Token 20 sees keys 19 and 20; key 20 alone, then both, have scores of -Inf."""
    lens = [50, 7] + [0] * empty
    x = ta.make(221, dtype, 4, 2, 64, lens, lens)
    x["q"][20, :, 5] = 1.0
    x["q"][[19, 21], :, 5] = 0.25
    clean = ta.both(x, lens, lens, 2, 0)
    for keys in ([20], [19, 20]):
        y = dict(x, k=x["k"].clone())
        y["k"][keys, :, 5] = -float("inf")
        got = ta.both(y, lens, lens, 2, 0)
        rows = torch.ones(57, dtype=torch.bool)
        rows[keys] = rows[21] = False
        for name in ("o", "lse", "dq"):
            assert torch.equal(got[name][rows.cuda()], clean[name][rows.cuda()]), name
        if len(keys) == 1:                       # what is left is key 19
            u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -22
            v = x["v"][19].repeat_interleave(2, dim=0).float()
            assert ((got["o"][20].float() - v).abs() <= 2 * u * v.abs()).all()
        else:
            assert (got["o"][20] == 0).all() and torch.isneginf(got["lse"][20]).all()
            assert torch.isnan(got["dq"][20].float()).any(dim=-1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sequences,new", [(2, 1), (2, 3), (90, 20)])
def test_paged(dtype, sequences, new):
    """The decode kernel, and with many rows the forward kernel over a cache: the last
    token's one key has a score of -Inf."""
    lens = [40] * sequences
    x = td.make(222, dtype, 8, 4, 64, 16, lens, [new] * sequences, poison=False)
    last = torch.arange(sequences) * new + new - 1
    x["q"][last, :, 5] = 1.0
    clean = [t.clone() for t in td.run(x, 1, 0)]
    x["k"][x["table"][:, 2].long(), 39 % 16, :, 5] = -float("inf")
    o, lse = td.run(x, 1, 0)
    assert (o[last] == 0).all() and torch.isneginf(lse[last]).all()
    rest = torch.ones(len(o), dtype=torch.bool)
    rest[last] = False
    assert torch.equal(o[rest.cuda()], clean[0][rest.cuda()]) and torch.equal(lse[rest.cuda()], clean[1][rest.cuda()])
