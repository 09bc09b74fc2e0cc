"""dflash2_attend where one number of a value, and of nothing else, is a NaN or an infinity: every token that sees the key
has no finite number in that place, and no other token's result knows of it.

The keys lie in tiles that some query rows see whole and others do not: blocks of more rows than a warp (16 tokens of 5
heads) and than a stream (64 of 4), over a tile's end, before a window, and behind a shared prefix that some sequences see
whole and others do not.  Tolerance of the others as in test_gpu_attend.py."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_attend import CACHES, Case  # noqa: E402

pytestmark = pytest.mark.gpu
DIM = 3


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


def check(c, at, what, causal=True, window=0):
    """at: (sequence, position) of the spoilt values (in all heads)."""
    want, mag = c.reference(c.d ** -0.5, causal, window)
    for s, p in at:
        c.dev["v"][c.table[0 if p < c.shared else s, p // c.page], p % c.page, :, DIM] = \
            float("nan") if c.cache_type == "e4m3" else float(what)
    got = c.run(causal=causal, window=window)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -16 if c.cache_type == "e4m3" else 2.0 ** -14) * mag + 1e-30
    seeing = 0
    for s, n in enumerate(c.count):
        for t in range(n):
            hi = c.lens[s] - (n - 1 - t) if causal else c.lens[s]
            lo = max(0, hi - window) if window else 0
            if any(lo <= p < hi and (p < c.shared or x == s) for x, p in at):
                seeing += 1
                assert not np.isfinite(got[s, t, :, DIM]).any(), (s, t)
            else:
                assert (np.abs(got[s, t] - want[s, t]) <= tol[s, t]).all(), (s, t)
    assert seeing


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("nq,nkv,n_tok,length,at", [
    (5, 1, 16, 132, [120]), (5, 1, 16, 132, [127]), (10, 2, 16, 8200, [8186]), (10, 2, 16, 8200, [8191, 8192]),
    (4, 1, 64, 260, [200]), (4, 1, 64, 260, [255]), (4, 1, 64, 260, [0]), (4, 1, 16, 144, [127]), (2, 1, 20, 140, [125])])
def test_a_blocks_own_values_at_a_tiles_end(B, cache, what, nq, nkv, n_tok, length, at):
    c = Case(B, cache, 128, 16, nq, nkv, n_tok, [length, 40 + n_tok], seed=40 + length)
    check(c, [(0, p) for p in at], what)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("nq,nkv,n_tok,length,window,at", [
    (5, 1, 16, 300, 100, [186, 187, 199]), (4, 1, 64, 400, 130, [215]), (4, 1, 64, 400, 130, [300]),
    (5, 1, 16, 272, 129, [130]), (5, 1, 16, 272, 129, [128])])
def test_windows(B, cache, nq, nkv, n_tok, length, window, at):
    check(Case(B, cache, 128, 16, nq, nkv, n_tok, [length], seed=41), [(0, p) for p in at], "nan", window=window)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("nq,nkv,n_tok,lens,shared,at,causal", [
    (4, 1, 8, [100, 400, 350, 300], 256, [(1, 20)], True), (4, 1, 8, [100, 400, 350, 300], 256, [(1, 120)], True),
    (5, 1, 16, [60, 300, 300, 300], 128, [(0, 70)], False), (4, 1, 8, [300] * 40 + [70], 256, [(0, 100)], True),
    (8, 2, 8, [500, 260, 400, 450], 256, [(0, 255), (2, 300)], True)])
def test_a_prefix_that_not_all_sequences_see_whole(B, cache, nq, nkv, n_tok, lens, shared, at, causal):
    check(Case(B, cache, 128, 16, nq, nkv, n_tok, lens, shared=shared, seed=42), at, "nan", causal=causal)


@pytest.mark.parametrize("cache", CACHES)
def test_ragged_blocks(B, cache):
    c = Case(B, cache, 128, 16, 5, 1, 20, [140, 300, 141], n_new=[16, 1, 20], seed=43)
    check(c, [(0, 126), (2, 127)], "nan")
