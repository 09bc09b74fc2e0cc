"""dflash2_attend with kv_len outside what the block table holds: below 0 it counts as 0, past the table as all of it, and
the other sequences of the call do not notice.  Both kernels, with more tokens than keys, a window and a shared prefix."""

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


@pytest.fixture(autouse=True, params=[1, 2], ids=["general", "tensor"])
def kernel(request, B):
    B.dflash2_test_force_attend(request.param)
    yield
    B.dflash2_test_force_attend(0)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("bad,counts_as", [(-1, 0), (-2 ** 31, 0), (20 * 16 + 1, 20 * 16), (2 ** 31 - 1, 20 * 16)])
@pytest.mark.parametrize("shared,causal,window", [(0, True, 0), (0, False, 70), (64, True, 0), (64, True, 100)])
def test_lengths_out_of_range(B, cache, d, bad, counts_as, shared, causal, window):
    c = Case(B, cache, d, 16, 8, 2, 5, [100, counts_as, 20 * 16], shared=shared, seed=90)
    assert c.table.shape[1] == 20
    want = c.check(causal=causal, window=window)
    c.lens[1] = bad
    assert np.array_equal(c.run(causal=causal, window=window, status=B.DEV_BAD_LENGTH), want)
    if counts_as == 0:
        assert not want[1].any()
