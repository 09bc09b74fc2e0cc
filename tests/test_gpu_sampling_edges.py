"""Sampling at the ends of its ranges, against the definition in float64
(tests/sampling_reference.py).  Tokens and kept sets are compared exactly;
a probability is good to 2^-20 relative (two ulp of the exponential, one of
its correction, one of the reciprocal, half a one of the product)."""

import numpy as np
import pytest

from tests import sampling_reference as R
from tests.helpers import lib

pytestmark = pytest.mark.gpu

RTOL = 2.0 ** -20


def settings_of(n, t, k, p, m):
    import torch
    f = lambda v, dt: None if v is None else torch.full((n,), v, dtype=dt, device="cuda")
    return f(t, torch.float32), f(k, torch.int32), f(p, torch.float32), f(m, torch.float32)


def draws(B, z, settings, u):
    import torch
    tok = torch.full((z.shape[0],), -7, dtype=torch.int32, device="cuda")
    B.dflash2_sample(z, *settings, torch.from_numpy(u).cuda(), tok)
    return tok.cpu().numpy()


def probs(B, z, settings):
    import torch
    out = torch.full((z.shape[0], 1, z.shape[1]), float("nan"), device="cuda")
    B.dflash2_target_probs(z[:, None], *settings, out)
    return out[:, 0].cpu().numpy()


@pytest.mark.parametrize("temp", [np.inf, 1e30])
@pytest.mark.parametrize("n_border", [2047, 2048, 2049])
def test_a_full_list_of_equal_masses_at_the_top_p_border(temp, n_border):
    """At such temperatures every token has the largest mass.  The border's
    tokens, as many as a list holds and all of them in one warp's part of the
    row (36000 bf16 logits, 200 rows: one CTA of 16 warps a row, 2250 tokens
    each), are two values of one bin; the draws go over all that is kept."""
    import torch
    B = lib()
    n, V, ahead = 200, 36000, 20000
    z = np.full(V, -63.0, np.float32)
    first = 11300                                   # in the range of warp 5: 11248 .. 13499
    border = np.arange(first, first + n_border)
    z[border] = np.where(np.arange(n_border) % 2, -1 / 32, 0.0)
    rest = np.setdiff1d(np.arange(V), border)
    z[np.random.default_rng(1).permutation(rest)[:ahead]] = 1.0
    p = np.float32((ahead + n_border - 0.5) / V)
    u = np.random.default_rng(2).random(n, dtype=np.float32)
    zt = torch.from_numpy(np.broadcast_to(z, (n, V)).copy()).cuda().to(torch.bfloat16)
    mass = R.masses(z, temp, 0, float(p))
    assert np.count_nonzero(mass) == ahead + n_border
    got = draws(B, zt, settings_of(n, temp, None, float(p), None), u)
    np.testing.assert_array_equal(got, [R.draw(mass, x) for x in u])
    pr = probs(B, zt[:2], settings_of(2, temp, None, float(p), None))
    np.testing.assert_allclose(pr, np.broadcast_to(mass / mass.sum(), (2, V)), rtol=RTOL)


@pytest.mark.parametrize("k,p", [(None, None), (4, None), (500, None), (None, 0.9), (500, 0.5)])
@pytest.mark.parametrize("m", [0.5, 1.0, 3.0])
def test_min_p_at_an_infinite_temperature_keeps_every_token(k, p, m):
    """Every mass is 1, so none is below min(min_p, 1)."""
    import torch
    B = lib()
    n, V = 4, 3001
    z = np.random.default_rng(3).standard_normal((n, V)).astype(np.float32)
    z[:, ::7] = -np.inf
    zt = torch.from_numpy(z).cuda()
    st = settings_of(n, np.inf, k, p, m)
    mass = [R.masses(z[r], np.inf, k or 0, 1.0 if p is None else float(np.float32(p)), m) for r in range(n)]
    got = probs(B, zt, st)
    for r in range(n):
        np.testing.assert_allclose(got[r], mass[r] / mass[r].sum(), rtol=RTOL)
    u = np.array([0.1, 0.4, 0.7, 0.99], np.float32)
    np.testing.assert_array_equal(draws(B, zt, st, u), [R.draw(mass[r], u[r]) for r in range(n)])


@pytest.mark.parametrize("k,p,m", [(None, None, None), (2, None, None), (150, None, None), (None, 0.6, None),
                                   (None, None, 0.5), (None, None, 1.0), (300, 0.5, 0.5)])
@pytest.mark.parametrize("temp", [1.0, 1e38, np.inf])
def test_infinite_logits_share_the_whole_mass_at_any_temperature(temp, k, p, m):
    import torch
    B = lib()
    V = 3001
    z = np.random.default_rng(4).standard_normal((1, V)).astype(np.float32)
    tops = [5, 1700, 2999]
    z[0, tops] = np.inf
    z[0, 9] = -np.inf
    zt = torch.from_numpy(z).cuda()
    kept = tops[:2] if k == 2 else tops
    if p is not None:
        kept = kept[:int(np.ceil(float(np.float32(p)) * len(kept)))]
    want = np.zeros(V)
    want[kept] = 1 / len(kept)
    st = settings_of(1, temp, k, p, m)
    np.testing.assert_allclose(probs(B, zt, st)[0], want, rtol=RTOL)
    for u in (0.0, 0.4, 0.9):
        assert draws(B, zt, st, np.array([u], np.float32))[0] == kept[int(float(np.float32(u)) * len(kept))]
