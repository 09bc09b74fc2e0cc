"""dflash2_adjust_logits records bad token ids and lengths whatever the settings are: with penalties left out, neutral in
one sequence and not in another, and with nothing but a mask.  The rows of a neutral sequence stay as they are, bit by
bit."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_adjust import Case, dev  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_speculative_decoding_dflash2_gb300 import binding
    binding.lib()
    return binding


def neutral(dtype, history, vocab=5000, rows=4, seed=50):
    c = Case(3, rows, vocab, dtype, history, seed=seed)
    c.n[:] = history
    c.prompt[:] = 0
    c.rho[:], c.presence[:], c.frequency[:] = 1, 0, 0
    return c


LEFT_OUT = dict(repetition=None, presence=None, frequency=None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("over", [LEFT_OUT, {}], ids=["left out", "neutral"])
@pytest.mark.parametrize("history", [10, 7000])
def test_neutral_settings(B, dtype, over, history):
    c = neutral(dtype, history)
    z = c.z.double().numpy()
    assert np.array_equal(c.run(B, **over), z)
    for bad in (5000, 2 ** 31 - 1, -1, -2 ** 31):
        for at in ((0, 0), (2, history - 1), (1, history // 2)):
            keep = c.tokens[at]
            c.tokens[at] = bad
            assert np.array_equal(c.run(B, status=B.DEV_BAD_TOKEN, **over), z)
            c.tokens[at] = keep
    for bad in (5000, -2):
        c.path[1, 2] = bad
        assert np.array_equal(c.run(B, status=B.DEV_BAD_TOKEN, **over), z)
    c.path[1, 2] = -1  # (no token)
    assert np.array_equal(c.run(B, **over), z)
    for bad in (history + 1, -1):
        c.n[1] = bad
        assert np.array_equal(c.run(B, status=B.DEV_BAD_LENGTH, **over), z)
    c.n[1] = 3  # ids behind a sequence's tokens are not looked at
    c.tokens[1, 3:] = -7
    assert np.array_equal(c.run(B, **over), z)


def test_one_sequence_of_several(B):
    c = neutral(torch.float32, 40)
    c.presence[0] = 1.0
    good = c.check(B)
    c.tokens[2, 5] = 10 ** 6
    assert np.array_equal(c.run(B, status=B.DEV_BAD_TOKEN), good)
    c.n[1] = 41
    assert np.array_equal(c.run(B, status=B.DEV_BAD_TOKEN | B.DEV_BAD_LENGTH), good)


def test_a_path_without_tokens(B):
    c = neutral(torch.float32, 5)
    c.path[0, 0] = 5000
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    z = c.z.cuda()
    out = torch.empty_like(z)
    B.dflash2_adjust_logits(z, None, None, out, path=dev(c.path, torch.int32), workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, z) and B.dflash2_read_device_status(ws) == B.DEV_BAD_TOKEN
