"""Query rows that are not finite where the walk of a key tile ends.  The last tile of
rows of a walk is seldom full, and what stands behind its last row must not carry that
row's NaN or Inf to keys that the row does not see.

A walk ends at the last row that sees the last key of a tile of 16 or 64 keys, and at
the sequence's last row.  Both forms of the kernels (see test_gpu_window_forms.py)."""
import pytest
import torch

import test_gpu_window_attention as ta

pytestmark = pytest.mark.gpu
H, HK, D = 6, 3, 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ends(n, off, window):
    """Rows of a sequence of n queries, the first at position off, that end a walk."""
    rows = {n - 1} | {key0 + keys + window - 2 - off for keys in (16, 64) for key0 in (0, 64, 128)}
    return sorted(i for i in rows if 0 <= i < n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("empty", [0, 600], ids=["split", "whole"])
@pytest.mark.parametrize("n,prefix,window,sinks", [(300, 0, 128, 0), (300, 0, 100, 4), (215, 0, 10, 0), (200, 70, 61, 20),
                                                   (700, 0, 33, 64)])
@pytest.mark.parametrize("what", ["q", "d_o"])
def test_rows_that_end_a_walk(dtype, empty, n, prefix, window, sinks, what):
    """NaN in a row of the first key head's group, Inf in one of the second's: the keys
    that the row sees get gradients that are not finite, all others and all other rows
    the ones they have without."""
    first = 40                                   # tokens of a sequence before
    lens_q, lens_k = [first, n, 25] + [0] * empty, [first, n + prefix, 25] + [0] * empty
    x = ta.make(201, dtype, H, HK, D, lens_q, lens_k)
    clean = ta.both(x, lens_q, lens_k, window, sinks)
    row, key = torch.arange(sum(lens_q), device="cuda"), torch.arange(sum(lens_k), device="cuda") - first
    bad = ends(n, prefix, window)
    assert len(bad) >= 3
    for i in bad:
        y = dict(x, **{what: x[what].clone()})
        y[what][first + i, 0] = float("nan")
        y[what][first + i, 2] = float("inf")
        got = ta.both(y, lens_q, lens_k, window, sinks)
        p = i + prefix
        seen = (key >= 0) & (key <= p) & ((p - key < window) | (key < sinks))
        for name in ("dk", "dv"):
            leaked = (got[name] != clean[name]).any(-1)[~seen].any(-1).nonzero().flatten()
            assert not len(leaked), f"{name}, row {i}: keys {key[~seen][leaked].tolist()}"
            assert torch.equal(got[name][:, 2], clean[name][:, 2])
            assert not torch.isfinite(got[name][seen][:, :2]).any(), f"{name}, row {i}"
        for name in ("o", "lse", "dq"):
            rest = row != first + i
            assert torch.equal(got[name][rest], clean[name][rest]), f"{name}, row {i}"
            assert torch.equal(got[name][~rest][:, [1, 3, 4, 5]], clean[name][~rest][:, [1, 3, 4, 5]]), f"{name}, row {i}"
        assert not torch.isfinite(got["dq"][first + i, [0, 2]]).any()
