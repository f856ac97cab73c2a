"""Gradients of short documents, alone and beside long ones (bf16)."""
import pytest
import torch

import test_gpu_window_attention as ta
import window_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("empty", [0, 600], ids=["split", "whole"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("short,long", [([8] * 30, [1000]), ([31, 5, 17] * 4, [700, 300]), ([8] * 30, [])])
@pytest.mark.parametrize("window,sinks", [(50, 0), (400, 4)])
def test_short_documents_beside_long_ones(empty, d, short, long, window, sinks):
    """Rows that see at most 32 keys, all of their document's: dq is off by its own rounding
    alone, at most 2^-8 of a value, with mantissas spread evenly in the logarithm 2^-8 /
    sqrt(3) sqrt(0.54) = 1.66e-3 in the norm, and a fifth more for all else.  (With
    the error of a delta from the rounded o: 2.8e-3.)  The long documents' first 32
    tokens are such rows too."""
    lens = short[:len(short) // 2] + long + short[len(short) // 2:] + [0] * empty
    x = ta.make(211, "bf16", 16, 4, d, lens, lens)
    got = ta.both(x, lens, lens, window, sinks)
    want, _ = ref.attention(x["q"], x["k"], x["v"], lens, lens, window, sinks, d_o=x["d_o"])["dq"]
    place = torch.cat([torch.arange(n) for n in lens])
    size = torch.cat([torch.full((n,), n) for n in lens])
    off = got["dq"].double().cpu() - want
    for name, rows in (("short", size <= 32), ("first of long", (size > 32) & (place < 32))):
        if rows.any():
            err = float(off[rows].norm() / want[rows].norm())
            print(f"[window] dq, {name}: {err:.2e}", flush=True)
            assert err <= 2.0e-3, name


@pytest.mark.parametrize("empty", [0, 600], ids=["split", "whole"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (16, 4)])
@pytest.mark.parametrize("short,long", [([8] * 30, [1000]), ([31, 5, 17, 32] * 4, [700, 300]), ([1, 3, 2, 4, 9, 5] * 4, [])])
def test_keys_that_few_rows_see(empty, d, H, Hk, short, long):
    """dk and dv of documents of at most 32 tokens: few weights make them, so that a
    rounding of each would show (2.3e-3 in the norm, and up to 2.6e-3 in a small batch).  As
    for dq above: their own rounding, 1.66e-3, and a fifth more."""
    lens = short[:len(short) // 2] + long + short[len(short) // 2:] + [0] * empty
    x = ta.make(212, "bf16", H, Hk, d, lens, lens)
    got = ta.both(x, lens, lens, 500, 4)
    want = ref.attention(x["q"], x["k"], x["v"], lens, lens, 500, 4, d_o=x["d_o"])
    size = torch.cat([torch.full((n,), n) for n in lens])
    for name in ("dk", "dv"):
        value = want[name][0][size <= 32]
        err = float((got[name].double().cpu()[size <= 32] - value).norm() / value.norm())
        print(f"[window] {name}: {err:.2e}", flush=True)
        assert err <= 2.0e-3, name
