"""dflash2_adjust_logits refuses token buffers whose indexes would pass 32 bits in a block's walk.  On the host, before
anything is launched, so without a GPU, on addresses that are never read."""

import pytest

P = 1 << 20


@pytest.mark.parametrize("most", [2 ** 31 - 1, 2 ** 31 - 2048, 2 ** 31 - 4095])
def test_buffers_near_two_to_the_31(most):
    pytest.importorskip("torch")
    from block_speculative_decoding_dflash2_gb300 import binding
    try:
        f = binding.lib().dflash2_adjust_logits
    except ImportError as e:
        pytest.skip(str(e))
    assert f(0, 2, 3, 10, P, 10, P, most, P, None, None, None, None, None, None, None, 0, None, P, 10, None, None) == -2
