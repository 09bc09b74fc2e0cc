"""What dflash2_attend makes of 8-bit rows where coarser arithmetic shows.

The general kernel keeps queries, weights and sums in fp32, whatever the pages' size: 2^-14 of the sum of weight times
|value| (scores' errors, as in test_gpu_attend.py) beside the result's own rounding of 2^-8.

On the tensor cores a weight times its value's scale is rounded to 11 bits (2^-11), which its three codes hold exactly, but
for what lies below 2^-27 of the row's largest."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_attend import CACHES, Case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_speculative_decoding_dflash2_gb300 import binding
    binding.lib()
    return binding


@pytest.fixture
def force(B):
    yield B.dflash2_test_force_attend
    B.dflash2_test_force_attend(0)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("page", [16, 48, 20])
@pytest.mark.parametrize("nq,nkv,n_tok,lens,shared,window", [
    (8, 2, 8, [8, 20, 130, 257], 0, 0), (5, 1, 3, [700, 90], 0, 100), (8, 1, 2, [300, 310, 500], 240, 0),
    (2, 2, 1, [1200], 0, 0)])
def test_the_general_kernel_keeps_fp32(B, force, cache, d, page, nq, nkv, n_tok, lens, shared, window):
    force(1)
    c = Case(B, cache, d, page, nq, nkv, n_tok, lens, shared=shared, seed=60)
    got = c.run(window=window)
    want, mag = c.reference(d ** -0.5, True, window)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * mag + 1e-30).all()


@pytest.mark.parametrize("spread", [0, 12])
def test_weights_that_cancel(B, force, spread):
    """A few keys with values of +1 and -1 (or by powers of two smaller): what their weights' codes leave out shows.  Ten
    thousand rows of 2 to 9 keys; beside the weights' 2^-11, 2^-15 for the scores' errors (2^-16, as in
    test_gpu_attend.py), the sums' and what 9 keys lose below 2^-27 of the largest."""
    force(2)
    c = Case(B, "e4m3", 128, 16, 32, 1, 8, [9] * 40, seed=64)
    for s in range(40):
        for p in range(9):
            c.pool["v"][c.table[s, 0], p] = (1.0 if p % 2 else -1.0) * 2.0 ** (-(p * 7 % 5) * spread // 5)
    c.quantise()
    got = c.run()
    want, mag = c.reference(128 ** -0.5, True, 0)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -15) * mag).all()
