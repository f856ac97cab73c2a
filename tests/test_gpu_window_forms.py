"""The two forms of the window kernels that small batches choose between: waves that
share 16 rows (or keys) and split their walk, and waves with rows of their own.  Which one runs follows from the sizes and the number of
sequences, so that 600 empty sequences behind the others select the second
(window_common.h, split_waves; the launch of dk and dv in window_backward.hip)."""
import pytest
import torch

import test_gpu_window_attention as ta
import test_gpu_window_decode as td
import window_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", ["f32", "bf16"])
FORMS = pytest.mark.parametrize("empty", [0, 600], ids=["split", "whole"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@DTYPES
@FORMS
@pytest.mark.parametrize("H,Hk,d", [(3, 3, 128), (8, 2, 64), (5, 1, 128), (12, 3, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 4), (64, 0), (100, 64), (33, 17), (2 ** 31 - 1, 3)])
def test_ragged_batch(dtype, empty, H, Hk, d, window, sinks):
    lens = [1, 0, 63, 64, 65, 17, 129, 2, 200, 16] + [0] * empty
    x = ta.make(81, dtype, H, Hk, d, lens, lens)
    ta.check_all(f"{H}/{Hk} {d} W={window} S={sinks}", x, ta.both(x, lens, lens, window, sinks), lens, lens, window, sinks)


@DTYPES
@FORMS
@pytest.mark.parametrize("lens_q,lens_k", [([5, 1, 70, 0, 33], [40, 130, 70, 9, 300]), ([70, 130, 3], [20, 129, 0])])
@pytest.mark.parametrize("window,sinks", [(1, 0), (32, 2), (150, 64)])
def test_unequal_lengths(dtype, empty, lens_q, lens_k, window, sinks):
    lens_q, lens_k = lens_q + [0] * empty, lens_k + [0] * empty
    x = ta.make(82, dtype, 8, 2, 128, lens_q, lens_k)
    ta.check_all(f"W={window} S={sinks}", x, ta.both(x, lens_q, lens_k, window, sinks), lens_q, lens_k, window, sinks)


@DTYPES
@FORMS
@pytest.mark.parametrize("sinks", [1, 16, 17, 64])
def test_sinks_of_long_sequences(dtype, empty, sinks):
    """Pieces of the sinks' walk, for one to four key tiles with sinks."""
    lens = [2500, 90, 1200] + [0] * empty
    x = ta.make(83, dtype, 4, 2, 64, lens, lens)
    ta.check_all(f"S={sinks}", x, ta.both(x, lens, lens, 40, sinks), lens, lens, 40, sinks)


@FORMS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(30, 5), (1000, 0)])
def test_chunks_over_a_cache(empty, d, window, sinks):
    lens, new = [300, 100, 64, 129] + [0] * empty, [100, 100, 1, 65] + [0] * empty
    x = td.make(84, "f32", 8, 2, d, 16, lens, new)
    if empty:                  # more rows than the empty sequences have
        lens, new = [n + 700 for n in lens[:4]] + [1] * 40, [700] * 4 + [1] * 40
        x = td.make(85, "f32", 16, 4, d, 16, lens, new)
    # batches that take the kernel of chunks
    assert sum(new) * 4 > 16 * len(new) and (sum(new) * 4 // 16 + len(new)) * x["k"].shape[2] > 64
    td.check(f"{d} W={window} S={sinks}", x, lens, new, window, sinks)


@DTYPES
@FORMS
@pytest.mark.parametrize("what", ["q", "k", "v", "d_o"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_within_the_window(dtype, empty, what, value):
    """Token 80 of a sequence is not finite: rows and keys that do not see it are
    as without it."""
    lens, window, sinks = [150, 40] + [0] * empty, 20, 3
    x = ta.make(86, dtype, 4, 2, 64, lens, lens)
    clean = ta.both(x, lens, lens, window, sinks)
    x[what][80, 0] = value
    got = ta.both(x, lens, lens, window, sinks)
    i = torch.arange(190)
    if what in ("k", "v"):     # rows that see the key; the keys that those rows see
        rows = (i >= 80) & (i < 100)
        keys = (i < sinks) | ((i > 60) & (i < 100))
    else:
        rows = i == 80
        keys = (i < sinks) | ((i > 60) & (i <= 80))
    for name, touched in (("o", rows), ("lse", rows), ("dq", rows), ("dk", keys), ("dv", keys)):
        at = (~touched).cuda()
        assert torch.equal(got[name][at], clean[name][at]), name
    if what != "d_o":
        assert not torch.isfinite(got["o"][80]).all()


@DTYPES
@FORMS
def test_same_result_every_time(dtype, empty):
    lens = [1500, 30, 77] + [0] * empty
    x = ta.make(87, dtype, 8, 2, 64, lens, lens)
    first = ta.both(x, lens, lens, 100, 20)
    for _ in range(3):
        again = ta.both(x, lens, lens, 100, 20)
        assert all(torch.equal(first[n], again[n]) for n in first)


@DTYPES
def test_the_forms_agree(dtype):
    """Within the sum of both bounds: each is within its own of the formula."""
    lens = [700, 1, 64]
    x = ta.make(88, dtype, 8, 2, 128, lens, lens)
    a = ta.both(x, lens, lens, 150, 10)
    many = lens + [0] * 600
    b = ta.both(x, many, many, 150, 10)
    want = ref.attention(x["q"], x["k"], x["v"], lens, lens, 150, 10, d_o=x["d_o"])
    for name, (_, bound) in want.items():
        assert ((a[name].double() - b[name].double()).abs().cpu() <= 2 * bound).all(), name


@FORMS
@pytest.mark.parametrize("lens,window,sinks", [([200, 85, 50], 3, 0), ([300], 12, 4), ([8] * 30, 50, 0)])
def test_rows_that_see_few_keys(empty, lens, window, sinks):
    """dq in bf16 is off by its own rounding alone: at most 2^-8 of a value, with mantissas
    spread evenly in the logarithm 2^-8 / sqrt(3) sqrt(0.54) = 1.66e-3 in the norm, and
    a fifth more for all else.  (With the error of a delta from the rounded o: 2.8e-3.)"""
    lens = lens + [0] * empty
    x = ta.make(89, "bf16", 16, 4, 64, lens, lens)
    got = ta.both(x, lens, lens, window, sinks)
    want, _ = ref.attention(x["q"], x["k"], x["v"], lens, lens, window, sinks, d_o=x["d_o"])["dq"]
    err = float((got["dq"].double().cpu() - want).norm() / want.norm())
    print(f"[window] dq, window {window}: {err:.2e}", flush=True)
    assert err <= 2.0e-3
