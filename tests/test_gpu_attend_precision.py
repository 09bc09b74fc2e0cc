"""What dflash2_attend makes of 8-bit rows where coarser arithmetic shows.

The general kernel keeps queries, weights and sums in fp32, whatever the pages' size: 2^-14 of the sum of weight times
|value| (scores' errors, as in test_gpu_attend.py) beside the result's own rounding of 2^-8.

On the tensor cores a query row is held as two 8-bit codes a value: exactly for values down to 2^-13 of the row's largest,
within 2^-21 of the largest below that.  A score may be off by scale * sum of |error of q| |k|, at most E over the keys;
weights, relative to each other, by exp(2 E) - 1.  A weight times its value's scale is rounded to 11 bits (2^-11), which its
three codes hold exactly, but for what lies below 2^-27 of the row's largest."""

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


def flat_pool(c):
    for name in ("k", "v"):
        c.pool[name][:] = torch.where(torch.isnan(c.pool[name]), c.pool[name], torch.zeros_like(c.pool[name]))


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("cache", CACHES)
def test_small_channels_beside_a_large_one(B, force, cache, mode):
    """A query with one channel of 2^10, which no key has, and others of 1 and 1 + 2^-7: two keys whose scores differ by
    64 * 2^-7 * scale only.  Their mean is tanh of half that, which all of the queries' bits make."""
    force(mode)
    c = Case(B, cache, 128, 16, 2, 1, 2, [3], seed=61)
    flat_pool(c)
    c.q[:] = 0
    c.q[..., 1:64] = 1 + 2.0 ** -7
    c.q[..., 64:127] = 1
    c.q[..., 0] = 2.0 ** 10
    page = c.table[0, 0]
    # the last token sees three keys, the first one two
    c.pool["k"][page, 0, :, 1:64], c.pool["k"][page, 0, :, 64:127] = 1, -1
    c.pool["v"][page, 0], c.pool["v"][page, 1], c.pool["v"][page, 2] = 1, -1, 0
    c.quantise()
    got = c.run()
    want, _ = c.reference(128 ** -0.5, True, 0)
    assert 0.021 < want[0, 0, 0, 0] < 0.022
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 + 2.0 ** -16).all()


@pytest.mark.parametrize("high", [2.0 ** 6, 2.0 ** 10, 2.0 ** 14])
@pytest.mark.parametrize("nq,nkv,n_tok,lens", [(8, 2, 4, [5, 40, 300]), (5, 1, 16, [500, 30]), (4, 1, 64, [200])])
def test_channels_far_above_the_others(B, force, high, nq, nkv, n_tok, lens):
    """Two channels of a query far above its others, with keys that are as much smaller there."""
    force(2)
    c = Case(B, "e4m3", 128, 16, nq, nkv, n_tok, lens, seed=62)
    c.q[..., 5:7] = (c.q[..., 5:7].float() * high).to(torch.bfloat16)
    c.pool["k"][..., 5:7] = (c.pool["k"][..., 5:7].float() / high).to(torch.bfloat16)
    c.quantise()
    got = c.run()
    want, mag = c.reference(128 ** -0.5, True, 0)
    for s, n in enumerate(c.count):
        rows = [(c.table[s, p // 16], p % 16) for p in range(lens[s])]
        k = np.abs(np.array([c.vals["k"][r] for r in rows])).reshape(-1, nkv, 128)
        q = np.abs(c.q[s, :n].double().numpy())
        top = q.max(-1, keepdims=True)
        err = np.where(q >= 2.0 ** -13 * top, 0.0, 2.0 ** -21 * top)
        off = 128 ** -0.5 * np.einsum("thd,khd->thk", err, np.repeat(k, nq // nkv, 1)).max(-1)[..., None]
        tol = 2.0 ** -8 * np.abs(want[s, :n]) + (2.0 ** -9 + 2.0 ** -16 + np.expm1(2 * off)) * mag[s, :n]
        assert (np.abs(got[s, :n] - want[s, :n]) <= tol).all(), s


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("power", [-75, -60, 60, 100])
@pytest.mark.parametrize("nq,n_tok,lens", [(4, 3, [3, 140, 700]), (4, 64, [200])])
def test_values_of_any_size(B, force, cache, mode, power, nq, n_tok, lens):
    """All values of a head by the same power of two larger or smaller: so is the result.  (2^-75 is a scale of 2^-83 of
    8-bit rows.  The tensor cores then lose 2^-27 * 2^3 of the largest weight in each of up to 700 keys, less than 2^-12
    of the sum of weight times |value|, beside the 2^-11 of each weight.)"""
    force(mode)
    c = Case(B, cache, 128, 16, nq, 1, n_tok, lens, seed=63, spread=1.0)
    v = c.pool["v"].float()
    c.pool["v"] = (torch.sign(v) * torch.clamp(v.abs(), 0.5, 1.0) * 2.0 ** power).to(torch.bfloat16)
    c.quantise()
    got = c.run()
    want, mag = c.reference(128 ** -0.5, True, 0)
    wide = 2.0 ** -9 + 2.0 ** -16 if cache == "e4m3" and mode == 2 else 2.0 ** -14
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + wide * mag).all()


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
