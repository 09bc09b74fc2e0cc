"""dflash2_attend where the scales of keys and values lie far apart: keys that a token does not see with the largest codes
and exponents (or none that is a number), and a visible value far above the others behind a weight far below theirs.

Tolerance as in test_gpu_attend.py: 2^-8 of the value for its own rounding, and 2^-9 + 2^-16 (8-bit caches on the tensor
cores) or 2^-14 of the sum of weight times |value|.  None of it depends on what a token does not see, nor on how far the
scales of the values lie apart."""

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


@pytest.fixture(autouse=True, params=[0, 2], ids=["choice", "tensor"])
def kernel(request, B):
    """The library's choice of a kernel, and the tensor cores' for short sequences too."""
    B.dflash2_test_force_attend(request.param)
    yield
    B.dflash2_test_force_attend(0)


def spoil(c, page, slots, kind, names=("k", "v"), byte=None):
    """Overwrites positions of a page on the device: the largest finite numbers, or none."""
    for name in names:
        if c.cache_type == "bf16":
            c.dev[name][page, slots] = 1e38 if kind == "large" else float("nan")
        else:
            c.dev[name].view(torch.uint8)[page, slots] = 0x7e if kind == "large" else 0x7f
            c.dev[name + "_exp"][page, slots] = (254 if byte is None else byte) if kind == "large" else 255


def compare(c, want, mag, causal=True, window=0, skip=()):
    got = c.run(causal=causal, window=window)
    fast8 = c.cache_type == "e4m3" and c.d == 128 and c.page % 16 == 0
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -16 if fast8 else 2.0 ** -14) * mag + 1e-30
    ok = np.abs(got - want) <= tol
    for s, t in skip:
        ok[s, t] = True
    assert ok.all(), np.argwhere(~ok)[:5].tolist()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("kind", ["large", "nan"])
def test_before_a_window(B, cache, d, kind):
    c = Case(B, cache, d, 16, 8, 2, 2, [206, 77, 300], seed=20)
    want, mag = c.reference(d ** -0.5, True, 50)
    for i, n in enumerate(c.lens):
        for p in range(n - 1 - 50 - 20, n - 1 - 50):  # token 0 sees the keys from n - 51 on
            spoil(c, c.table[i, p // 16], p % 16, kind)
    compare(c, want, mag, window=50)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("kind", ["large", "nan"])
def test_behind_a_token(B, cache, d, kind):
    """The last token's own key and value: every other token's result is what it was."""
    c = Case(B, cache, d, 16, 8, 2, 6, [206, 128, 40], seed=21)
    want, mag = c.reference(d ** -0.5, True, 0)
    for i, n in enumerate(c.lens):
        spoil(c, c.table[i, (n - 1) // 16], (n - 1) % 16, kind)
    compare(c, want, mag, skip=[(i, 5) for i in range(3)])


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("kind", ["large", "nan"])
def test_own_page_that_holds_the_end_of_the_shared_prefix(B, cache, kind):
    """A sequence's own copy of the page in which the prefix ends: the prefix is read elsewhere."""
    c = Case(B, cache, 128, 16, 8, 2, 4, [300, 150, 90], shared=72, seed=22)
    want, mag = c.reference(128 ** -0.5, True, 0)
    used = set(c.table[c.table >= 0].tolist())
    spare = [p for p in range(c.pool["k"].shape[0]) if p not in used]
    for i, page in zip((1, 2), spare):
        old = int(c.table[i, 4])
        for name in ("k", "v") if cache == "bf16" else ("k", "v", "k_exp", "v_exp"):
            t = c.dev[name].view(torch.uint8) if c.dev[name].dtype == torch.float8_e4m3fn else c.dev[name]
            t[page] = t[old]
        spoil(c, page, slice(0, 8), kind)
        c.table[i, 4] = page
    compare(c, want, mag)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("lens,far", [([130], 60), ([700], 300), ([700], 699)])
def test_a_large_value_behind_a_small_weight(B, cache, lens, far):
    """Weight 2^-90 or less of the others', value 2^50 or so of theirs: it adds next to nothing."""
    c = Case(B, cache, 128, 16, 1, 1, 1, lens, seed=23)
    page, at = c.table[0, far // 16], far % 16
    q = c.q[0, 0, 0].float()
    c.pool["k"][page, at, 0] = (-q * (70.0 / (float(q @ q) * 128 ** -0.5))).to(torch.bfloat16)
    c.pool["v"][page, at, 0] *= 2.0 ** 50
    c.quantise()
    c.check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("step", [1, -1])
def test_large_values_under_rising_and_falling_scores(B, cache, d, step):
    """Scores from -30 to 30 along the keys, values of about 2^96: their weighted mean is far inside the range.  (Many
    sequences, so that one block has whole ones.)"""
    n, batch = 400, 48
    c = Case(B, cache, d, 16, 8, 8, 1, [n] * batch, seed=24)
    for i in range(batch):
        q = c.q[i, 0].double()
        unit = q / ((q * q).sum(-1, keepdim=True) * d ** -0.5)
        for p in range(n):
            z = step * (60.0 * p / (n - 1) - 30.0)
            c.pool["k"][c.table[i, p // 16], p % 16] = (unit * z).to(torch.bfloat16)
    c.pool["v"] *= 2.0 ** 96
    c.quantise()
    c.check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [128, 64])
def test_a_query_of_zeros_under_a_small_scale(B, cache, d):
    c = Case(B, cache, d, 16, 4, 2, 5, [40, 5, 300], seed=25)
    c.q[:, :, 1] = 0
    c.q[:, :, 2] *= 2.0 ** -120
    c.check(scale=1e-12)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5000, 320, 319])
def test_windows_as_long_as_anything(B, cache, d, window):
    """More tokens than keys too: the first of them see nothing."""
    c = Case(B, cache, d, 16, 4, 2, 8, [3, 8, 320], seed=26)
    c.check(window=window)
