"""The operators from a target's logits to tokens (dflash2_sample,
dflash2_target_probs, dflash2_verify_logits) against the definition in
float64 (tests/sampling_reference.py).

Tolerance of a probability: p = e / M with e from exp2f (2 ulp), a first-order
correction (1 ulp), the whole masses' sum M (good to 2^-35) rounded to fp32 as
a reciprocal (1 ulp) and the product (half an ulp): below 2^-20 relative, plus
the smallest normal float where e / M underflows.  Tokens, kept sets and
accepted lengths are compared exactly.
"""

import numpy as np
import pytest

import dflash2_synth as S
from tests import sampling_reference as R
from tests.helpers import lib

pytestmark = pytest.mark.gpu

RTOL, ATOL = 2.0 ** -20, 2.0 ** -126


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def logits_of(rows, V, kind, seed, dtype="f32"):
    """(torch logits [rows, V], their float64 values)."""
    import torch
    g = np.random.default_rng(seed)
    z = g.standard_normal((rows, V)).astype(np.float32)
    if kind == "peaked":
        z *= 1.2
        n = min(40, V)
        for r in range(rows):
            z[r, g.choice(V, n, replace=False)] = 15 - 1.2 * np.log(np.arange(1, n + 1))
    elif kind == "ties":
        z = g.integers(0, 5, (rows, V)).astype(np.float32)
    elif kind == "wide":
        z *= 12
    elif kind == "equal":
        z[:] = np.float32(-3.5)
    t = dev(z, torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t, t.double().cpu().numpy()


def settings_of(n, spec):
    import torch
    t, k, p, m = spec
    f = lambda v, dt: None if v is None else torch.full((n,), v, dtype=dt, device="cuda")
    return f(t, torch.float32), f(k, torch.int32), f(p, torch.float32), f(m, torch.float32)


def plain(spec):
    t, k, p, m = spec
    f32 = lambda v, d: d if v is None else float(np.float32(v))
    return f32(t, 1.0), (0 if k is None else k), f32(p, 1.0), f32(m, 0.0)


def run_probs(B, z, settings, ws=None):
    import torch
    out = torch.full(z.shape, float("nan"), device="cuda")
    B.dflash2_target_probs(z, *settings, out, ws)
    return out


def check_probs(got, mass):
    p = mass / mass.sum() if mass.sum() > 0 else mass
    assert (got[p == 0] == 0).all() and (got[p >= ATOL] > 0).all()
    np.testing.assert_allclose(got, p, rtol=RTOL, atol=ATOL)


def run_sample(B, z, settings, u, prob=True):
    import torch
    tok = torch.full((z.shape[0],), -7, dtype=torch.int32, device="cuda")
    pr = torch.full((z.shape[0],), float("nan"), device="cuda") if prob else None
    B.dflash2_sample(z, *settings, dev(u), tok, pr)
    return tok.cpu().numpy(), None if pr is None else pr.cpu().numpy()


SPECS = [(None, None, None, None), (0.7, None, None, None), (1.0, 20, 0.95, None), (1.0, None, 0.9, None),
         (0.8, 1, None, None), (1.3, 50, 0.999, 0.02), (1.0, None, None, 0.05), (0.0, 20, 0.5, None),
         (2.0, None, 0.3, None), (0.05, 300, None, None)]


@pytest.mark.parametrize("V", [1, 2, 3, 31, 33, 128, 129, 1000, 4099, 50257])
@pytest.mark.parametrize("spec", SPECS, ids=str)
def test_probs_and_draws_over_sizes_and_filters(V, spec):
    B = lib()
    for kind, dtype in (("peaked", "f32"), ("ties", "f32"), ("normal", "bf16")):
        rows = 3
        z, zv = logits_of(rows, V, kind, seed=V + len(kind), dtype=dtype)
        g = np.random.default_rng(V)
        u = g.random(rows, dtype=np.float32)
        got = run_probs(B, z[:, None], settings_of(rows, spec))[:, 0].cpu().numpy()
        tok, pr = run_sample(B, z, settings_of(rows, spec), u)
        for r in range(rows):
            w = R.masses(zv[r], *plain(spec))
            check_probs(got[r], w)
            assert tok[r] == R.draw(w, u[r]), (kind, r)
            np.testing.assert_allclose(pr[r], w[tok[r]] / w.sum(), rtol=RTOL)


@pytest.mark.parametrize("kind", ["wide", "equal", "ties", "normal"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k,p", [(1, 1.0), (2, 1.0), (777, 1.0), (2048, 1.0), (2049, 0.99), (0, 0.5), (0, 0.001),
                                 (9000, 0.9), (20000, 1.0), (0, 1 - 2.0 ** -24)])
def test_large_kept_sets_and_ties(kind, dtype, k, p):
    B = lib()
    V = 9001
    z, zv = logits_of(2, V, kind, seed=5, dtype=dtype)
    spec = (1.0, k, p, None)
    got = run_probs(B, z[:, None], settings_of(2, spec))[:, 0].cpu().numpy()
    u = np.array([0.31, 0.97], np.float32)
    tok, _ = run_sample(B, z, settings_of(2, spec), u, prob=False)
    for r in range(2):
        w = R.masses(zv[r], *plain(spec))
        check_probs(got[r], w)
        assert tok[r] == R.draw(w, u[r])


def test_per_row_settings_and_the_draws_ends():
    import torch
    B = lib()
    V, n = 2000, 64
    z, zv = logits_of(n, V, "peaked", seed=1)
    g = np.random.default_rng(2)
    t = np.where(g.random(n) < 0.2, 0, g.random(n) + 0.2).astype(np.float32)
    t[:4] = [np.nan, -1.0, np.inf, 1e-30]
    k = np.where(g.random(n) < 0.3, 0, g.integers(1, 100, n)).astype(np.int32)
    k[5:8] = [-3, 2 ** 31 - 1, V]
    p = np.where(g.random(n) < 0.3, 1, g.random(n)).astype(np.float32)
    p[8:12] = [0.0, -1.0, 2.0, 1e-30]
    m = np.where(g.random(n) < 0.3, 0, g.random(n) * 0.2).astype(np.float32)
    m[12:15] = [1.0, 3.0, -0.5]
    u = g.random(n, dtype=np.float32)
    u[15:21] = [0.0, 0.99999994, 1.0, -1.0, 7.0, 0.5]
    settings = dev(t), dev(k), dev(p), dev(m)
    tok, _ = run_sample(B, z, settings, u)
    got = run_probs(B, z[:, None], settings)[:, 0].cpu().numpy()
    for r in range(n):
        w = R.masses(zv[r], float(t[r]), int(k[r]), float(p[r]), float(m[r]))
        check_probs(got[r], w)
        assert tok[r] == R.draw(w, u[r]), r
    torch.cuda.synchronize()


def special_rows():
    inf, nan, low = np.inf, np.nan, np.finfo(np.float32).min
    V = 300
    rows = np.full((9, V), -inf, np.float32)
    rows[1, 17] = -2.0                                    # one token left
    rows[2] = np.random.default_rng(0).standard_normal(V)
    rows[2, ::3] = nan
    rows[2, 1::3] = -inf
    rows[3] = nan                                         # none
    rows[4] = 0.0
    rows[4, [5, 250]] = inf                               # share the mass
    rows[5] = low                                         # all masked by the lowest value: equal tokens
    rows[6] = low
    rows[6, [3, 9, 299]] = [1.0, 2.0, 1.5]
    rows[7] = np.where(np.arange(V) % 2, 0.0, -0.0)       # equal
    rows[8, :7] = [1e38, -1e38, 3e38, 2.9e38, low, 0, 1]
    return rows


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("spec", [(1.0, None, None, None), (1.0, 4, 0.9, None), (0.5, None, 0.7, 0.01),
                                  (0.0, None, None, None)], ids=str)
def test_masked_and_extreme_rows(dtype, spec):
    import torch
    B = lib()
    z = dev(special_rows(), torch.bfloat16 if dtype == "bf16" else torch.float32)
    zv = z.double().cpu().numpy()
    n, V = z.shape
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = run_probs(B, z[:, None], settings_of(n, spec), ws)[:, 0].cpu().numpy()
    assert B.dflash2_read_device_status(ws) == B.DEV_EMPTY_ROW
    u = np.linspace(0.05, 0.9, n).astype(np.float32)
    tok = torch.empty((n,), dtype=torch.int32, device="cuda")
    pr = torch.empty((n,), device="cuda")
    B.dflash2_sample(z, *settings_of(n, spec), dev(u), tok, pr, ws)
    assert B.dflash2_read_device_status(ws) == B.DEV_EMPTY_ROW
    tok, pr = tok.cpu().numpy(), pr.cpu().numpy()
    for r in range(n):
        w = R.masses(zv[r], *plain(spec))
        check_probs(got[r], w)
        assert tok[r] == R.draw(w, u[r]), r
        assert pr[r] == 0 if tok[r] < 0 else abs(pr[r] - w[tok[r]] / w.sum()) <= RTOL * pr[r]
    keep = [r for r in range(n) if len(R.order_of(zv[r]))]  # (the lowest fp32 value rounds to -inf in bf16)
    assert len(keep) == (7 if dtype == "f32" else 6)
    run_probs(B, z[keep][:, None], settings_of(len(keep), spec), ws)
    assert B.dflash2_read_device_status(ws) == 0


@pytest.mark.parametrize("spec", [(None, None, None, None), (None, 4, None, None), (None, 4, 0.9, 0.1),
                                  (None, None, 0.9, None), (None, 500, 0.9, None), (None, None, None, 0.1)], ids=str)
@pytest.mark.parametrize("temp", [1.4e-45, 1e-40, 2e-39, 1e-38, 1e-20, 1e20, 3.4e38, np.inf])
def test_temperatures_at_the_ends_of_their_range(temp, spec):
    """Subnormal ones leave the largest logit all the mass, infinite ones give every token the same."""
    B = lib()
    z, zv = logits_of(5, 3001, "normal", 77)
    spec = (temp,) + spec[1:]
    mass = [R.masses(zv[r], *plain(spec)) for r in range(5)]
    got = run_probs(B, z[:, None], settings_of(5, spec))[:, 0].cpu().numpy()
    for r in range(5):
        check_probs(got[r], mass[r])
    for u in (0.0, 0.37, 0.9999999):
        u = np.full(5, u, np.float32)
        tok, _ = run_sample(B, z, settings_of(5, spec), u)
        assert list(tok) == [R.draw(mass[r], u[r]) for r in range(5)]


def test_rows_masked_with_the_lowest_bf16_value():
    import torch
    B = lib()
    z = torch.full((2, 513), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16, device="cuda")
    z[1, 400], z[1, 12] = 0.5, 0.25
    zv = z.double().cpu().numpy()
    for spec in ((1.0, None, None, None), (0.7, 3, 0.9, None)):
        got = run_probs(B, z[:, None], settings_of(2, spec))[:, 0].cpu().numpy()
        for r in range(2):
            check_probs(got[r], R.masses(zv[r], *plain(spec)))


def test_borders_at_zero_and_among_its_neighbours():
    """Cuts whose last token is +0, -0 or a subnormal next to them."""
    B = lib()
    V = 3000
    tiny = np.float32(1.4e-45)
    z = np.random.default_rng(4).choice(np.array([0.0, -0.0, tiny, -tiny, 1.0, -1.0], np.float32), (3, V))
    zt = dev(z)
    u = np.array([0.2, 0.5, 0.95], np.float32)
    for spec in ((1.0, None, 0.5, None), (1.0, None, 0.8, None), (1.0, 900, None, None), (1.0, 1700, 0.9, None),
                 (1.0, 60, None, None), (1.0, 2400, 0.7, 0.5)):
        got = run_probs(B, zt[:, None], settings_of(3, spec))[:, 0].cpu().numpy()
        tok, _ = run_sample(B, zt, settings_of(3, spec), u, prob=False)
        for r in range(3):
            w = R.masses(z[r], *plain(spec))
            check_probs(got[r], w)
            assert tok[r] == R.draw(w, u[r])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("by_k", [False, True])
def test_borders_among_few_distinct_values(dtype, by_k):
    """Logits on a coarse grid: large ties, so that the first guess of a top-p border is often wrong."""
    import torch
    B = lib()
    rows, V = 400, 15000
    g = np.random.default_rng(31 + by_k)
    z = dev(np.rint(4 * g.standard_normal((rows, V))).astype(np.float32), torch.bfloat16 if dtype == "bf16" else torch.float32)
    zv = z.double().cpu().numpy()
    t, p = g.uniform(1.2, 2, rows).astype(np.float32), g.uniform(0.05, 1, rows).astype(np.float32)
    k = g.integers(101, 4000, rows).astype(np.int32) if by_k else np.zeros(rows, np.int32)
    settings = (dev(t), dev(k), dev(p), None)
    u = g.random(rows, dtype=np.float32)
    got = run_probs(B, z[:, None], settings)[:, 0].cpu().numpy()
    tok, _ = run_sample(B, z, settings, u)
    for r in range(rows):
        w = R.masses(zv[r], float(t[r]), int(k[r]), float(p[r]), 0.0)
        check_probs(got[r], w)
        assert tok[r] == R.draw(w, u[r]), r


def test_draws_of_wide_flat_rows_are_exact():
    """400 draws from 50257 nearly equal tokens: one part in 10^7 of error in
    the running sum would move several of them."""
    B = lib()
    n, V = 400, 50257
    z, zv = logits_of(n, V, "normal", seed=77)
    u = np.random.default_rng(3).random(n, dtype=np.float32)
    for spec in ((1.0, None, None, None), (0.6, None, 0.95, None)):
        tok, _ = run_sample(B, z, settings_of(n, spec), u, prob=False)
        want = [R.draw(R.masses(zv[r], *plain(spec)), u[r]) for r in range(n)]
        np.testing.assert_array_equal(tok, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [151936, 1048576, 1048573])
@pytest.mark.parametrize("spec", [(1.0, 20, 0.95, None), (1.0, None, 0.9, None), (0.9, None, None, None)], ids=str)
def test_large_vocabularies(dtype, V, spec):
    B = lib()
    for kind in ("peaked", "normal"):
        z, zv = logits_of(2, V, kind, seed=9, dtype=dtype)
        u = np.array([0.123, 0.98], np.float32)
        got = run_probs(B, z[:, None], settings_of(2, spec))[:, 0].cpu().numpy()
        tok, _ = run_sample(B, z, settings_of(2, spec), u)
        for r in range(2):
            w = R.masses(zv[r], *plain(spec))
            check_probs(got[r], w)
            assert tok[r] == R.draw(w, u[r])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (5, 3), (8, 4)])
def test_row_strides_and_unaligned_rows(dtype, pad, shift):
    """Rows of a wider buffer, starting at any element; what lies between the
    rows is NaN and +inf and must not be read as logits."""
    import torch
    B = lib()
    n, V = 6, 1237
    src, _ = logits_of(n, V, "peaked", seed=4, dtype=dtype)
    buf = torch.full((n * (V + pad) + shift + 8,), float("nan"), dtype=src.dtype, device="cuda")
    buf[1::2] = float("inf")
    z = buf[shift:shift + n * (V + pad)].view(n, V + pad)[:, :V]
    z.copy_(src)
    u = np.random.default_rng(6).random(n, dtype=np.float32)
    st = settings_of(n, (1.0, 20, 0.95, None))
    assert torch.equal(run_probs(B, z[:, None], st), run_probs(B, src[:, None], st))
    np.testing.assert_array_equal(run_sample(B, z, st, u)[0], run_sample(B, src, st, u)[0])


def test_many_rows():
    B = lib()
    n, V = 70000, 5
    z, zv = logits_of(n, V, "normal", seed=8)
    u = np.random.default_rng(1).random(n, dtype=np.float32)
    tok, _ = run_sample(B, z, (None,) * 4, u)
    e = np.exp(zv - zv.max(1, keepdims=True))
    c = np.cumsum(e, 1)
    np.testing.assert_array_equal(tok, (c <= u[:, None].astype(np.float64) * c[:, -1:]).sum(1))


# ------------------------------------------------------------- verification

def verify_inputs(b, B_, V, kind, seed, dtype="f32", agree=0.75):
    import torch
    z, zv = logits_of(b * B_, V, kind, seed, dtype)
    z, zv = z.view(b, B_, V), zv.reshape(b, B_, V)
    g = np.random.default_rng(seed + 1)
    best = np.argmax(zv[:, :-1], axis=2)
    path = np.where(g.random(best.shape) < agree, best, g.integers(0, V, best.shape)).astype(np.int32)
    return z, zv, path, g.random((b, B_ - 1), dtype=np.float32), g.random(b, dtype=np.float32)


def run_verify(B, z, path, n_draft, settings, ua, u, seq=None, counters=None, ws=None):
    import torch
    b, B_, _ = z.shape
    full = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")
    a, out, n, nxt = full(b), full(b, B_), full(b), full(b)
    if ws is None:
        ws = torch.zeros(B.dflash2_verify_logits_workspace(b, B_), dtype=torch.uint8, device="cuda")
    B.dflash2_verify_logits(dev(path), None if n_draft is None else dev(n_draft), z, *settings, dev(ua), dev(u), a,
                            out, n, nxt, ws, seq, counters)
    return [t.cpu().numpy() for t in (a, out, n, nxt)]


def check_verify(got, zv, path, n_draft, per_seq, ua, u):
    a, out, n, nxt = got
    B_ = zv.shape[1]
    for s in range(zv.shape[0]):
        nd = B_ - 1 if n_draft is None else min(max(int(n_draft[s]), 0), B_ - 1)
        want, tok = R.verify(zv[s], path[s], nd, per_seq(s), ua[s], u[s])
        assert (a[s], n[s], nxt[s]) == (want, want + 1, tok), s
        assert list(out[s]) == list(path[s, :want]) + [tok] + [-1] * (B_ - 1 - want)


@pytest.mark.parametrize("V", [2, 33, 1000, 40003])
@pytest.mark.parametrize("spec", SPECS, ids=str)
@pytest.mark.parametrize("B_", [2, 8, 32])
def test_verify_against_the_definition(V, spec, B_):
    B = lib()
    b = 4
    for kind, dtype in (("peaked", "f32"), ("normal", "bf16")):
        z, zv, path, ua, u = verify_inputs(b, B_, V, kind, V + B_, dtype)
        got = run_verify(B, z, path, None, settings_of(b, spec), ua, u)
        check_verify(got, zv, path, None, lambda s: plain(spec), ua, u)


def test_verify_with_draft_counts_bad_tokens_and_counters():
    import torch
    B = lib()
    b, B_, V = 9, 6, 500
    z, zv, path, ua, u = verify_inputs(b, B_, V, "peaked", 31, agree=0.9)
    nd = np.array([0, 1, 2, 3, 4, 5, -4, 99, 5], np.int32)
    path[5, 0], path[8, 1] = -1, V  # not tokens: never accepted, nothing removed
    spec = (0.9, 20, 0.95, None)
    seq = dev(np.arange(b).astype(np.int32))
    cnt = torch.zeros((4 + 2 * B_ - 1,), dtype=torch.int64, device="cuda")
    got = run_verify(B, z, path, nd, settings_of(b, spec), ua, u, seq, cnt)
    check_verify(got, zv, path, nd, lambda s: plain(spec), ua, u)
    a = got[0]
    kept = np.clip(nd, 0, B_ - 1)
    np.testing.assert_array_equal(seq.cpu().numpy(), np.arange(b) + a + 1)
    c = cnt.cpu().numpy()
    assert list(c[:4]) == [b, kept.sum(), a.sum(), (kept - a).sum()]
    np.testing.assert_array_equal(c[4:4 + B_], np.bincount(a, minlength=B_))
    np.testing.assert_array_equal(c[4 + B_:], [(a > i).sum() for i in range(B_ - 1)])


def test_rows_past_the_drafts_are_not_read():
    B = lib()
    b, B_, V = 3, 5, 64
    z, zv, path, ua, u = verify_inputs(b, B_, V, "peaked", 41)
    nd = np.array([0, 2, 4], np.int32)
    for s in range(b):
        z[s, nd[s] + 1:] = float("nan")
    import torch
    ws = torch.zeros(B.dflash2_verify_logits_workspace(b, B_), dtype=torch.uint8, device="cuda")
    got = run_verify(B, z, path, nd, (None,) * 4, ua, u, ws=ws)
    check_verify(got, zv, path, nd, lambda s: (1.0, 0, 1.0, 0.0), ua, u)
    assert B.dflash2_read_device_status(ws) == 0


def test_verify_of_empty_rows_and_point_masses():
    import torch
    B = lib()
    b, B_, V = 3, 3, 40
    z = torch.full((b, B_, V), float("-inf"), device="cuda")
    z[1, 0, 7], z[1, 1, 8], z[1, 2, 9] = 0.0, 1.0, 2.0   # certain drafts
    z[2, 0, 5] = 3.0                                     # the draft 4 has no mass
    path = np.array([[1, 2], [7, 8], [4, 4]], np.int32)
    ua = np.array([[0, 0], [0.99999994, 1.0], [0, 0]], np.float32)
    ws = torch.zeros(B.dflash2_verify_logits_workspace(b, B_), dtype=torch.uint8, device="cuda")
    a, out, n, nxt = run_verify(B, z, path, None, (None,) * 4, ua, np.full(b, 0.5, np.float32), ws=ws)
    assert list(a) == [0, 2, 0] and list(nxt) == [-1, 9, 5]
    assert [list(o) for o in out] == [[-1, -1, -1], [7, 8, 9], [5, -1, -1]]
    assert B.dflash2_read_device_status(ws) == B.DEV_EMPTY_ROW


def test_greedy_is_verify_accept_of_the_largest_logits():
    import torch
    B = lib()
    b, B_, V = 16, 8, 1000
    z, zv, path, ua, u = verify_inputs(b, B_, V, "peaked", 51, "bf16", agree=0.9)
    st = settings_of(b, (0.0, None, None, None))
    a, out, n, nxt = run_verify(B, z, path, None, st, ua, u)
    e = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    ra, ro, rn, rx = e(b), e(b, B_), e(b), e(b)
    B.dflash2_verify_accept(b, B_, dev(path), dev(np.argmax(zv, 2).astype(np.int32)), ra, ro, rn, rx)
    for x, y in ((a, ra), (out, ro), (n, rn), (nxt, rx)):
        np.testing.assert_array_equal(x, y.cpu().numpy())


def test_one_workspace_serves_calls_of_any_size():
    """Batches around the size from which the rows are joined by a kernel of
    their own, and block sizes in any order, on one workspace."""
    import torch
    B = lib()
    ws = torch.zeros(B.dflash2_verify_logits_workspace(600, 32), dtype=torch.uint8, device="cuda")
    for b, B_ in ((2, 32), (257, 2), (256, 3), (600, 5), (1, 2), (255, 8), (7, 32), (300, 4)):
        z, zv, path, ua, u = verify_inputs(b, B_, 37, "peaked", b + B_)
        nd = np.random.default_rng(b).integers(0, B_, b).astype(np.int32)
        got = run_verify(B, z, path, nd, settings_of(b, (1.0, 5, 0.95, None)), ua, u, ws=ws)
        check_verify(got, zv, path, nd, lambda s: (1.0, 5, float(np.float32(0.95)), 0.0), ua, u)


@pytest.mark.parametrize("n", [255, 256, 257, 300, 1000, 2047, 2048])
@pytest.mark.parametrize("p,m", [(None, None), (0.8, None), (0.8, 0.3), (None, 0.3)])
def test_lists_around_their_sizes(n, p, m):
    """Kept sets around the list that is ranked, the one that is sorted and the
    largest one, draws and drafts among them."""
    B = lib()
    V, b, B_ = 7001, 5, 2
    z, zv, path, ua, u = verify_inputs(b, B_, V, "normal", n, agree=0.5)
    spec = (0.7, n, p, m)
    got = run_probs(B, z, settings_of(b, spec)).cpu().numpy()
    for s in range(b):
        for i in range(B_):
            check_probs(got[s, i], R.masses(zv[s, i], *plain(spec)))
    check_verify(run_verify(B, z, path, None, settings_of(b, spec), ua, u), zv, path, None, lambda s: plain(spec), ua, u)


@pytest.mark.parametrize("spec", [(1.0, 20, 0.95, None), (0.8, None, 0.9, 0.01)], ids=str)
def test_verify_logits_is_target_probs_then_verify_sampled(spec):
    import torch
    B = lib()
    b, B_, V = 12, 8, 6007
    z, zv, path, ua, u = verify_inputs(b, B_, V, "peaked", 61)
    st = settings_of(b, spec)
    got = run_verify(B, z, path, None, st, ua, u)
    p = run_probs(B, z, st)
    e = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    a, out, n, nxt = e(b), e(b, B_), e(b), e(b)
    B.dflash2_verify_sampled(b, B_, V, dev(path), None, p, dev(ua), dev(u), a, out, n, nxt)
    for x, y in zip(got, (a, out, n, nxt)):
        np.testing.assert_array_equal(x, y.cpu().numpy())


def test_sampled_verification_keeps_the_targets_distribution():
    """The first emitted token of 40000 verifications of one draft has the
    row's distribution: each frequency within 5 standard deviations."""
    import torch
    B = lib()
    n, V = 40000, 6
    row = np.array([1.0, 0.2, -0.5, 2.0, -np.inf, 0.1], np.float32)
    z = dev(np.broadcast_to(row, (n, 2, V)).copy())
    g = np.random.default_rng(12)
    path = g.choice([0, 3, 4], (n, 1), p=[0.3, 0.6, 0.1]).astype(np.int32)
    a, out, _, _ = run_verify(B, z, path, None, settings_of(n, (0.9, 4, None, None)), g.random((n, 1), dtype=np.float32),
                              g.random(n, dtype=np.float32))
    w = R.masses(row, float(np.float32(0.9)), 4)
    p = w / w.sum()
    f = np.bincount(out[:, 0], minlength=V) / n
    assert np.all(np.abs(f - p) <= 5 * np.sqrt(p * (1 - p) / n) + 1e-12)
    torch.cuda.synchronize()


# ------------------------------------------------- streams, graphs, repeats

def test_another_stream_a_captured_graph_and_two_graphs_sharing_a_workspace():
    import torch
    B = lib()
    b, B_, V = 3, 8, 5003
    z, zv, path, ua, u = verify_inputs(b, B_, V, "peaked", 71)
    z2, zv2, path2, ua2, u2 = verify_inputs(b, B_, V, "normal", 72)
    st = settings_of(b, (1.0, 20, 0.95, None))
    want = run_verify(B, z, path, None, st, ua, u)
    want2 = run_verify(B, z2, path2, None, st, ua2, u2)
    ws = torch.zeros(B.dflash2_verify_logits_workspace(b, B_), dtype=torch.uint8, device="cuda")
    buf = [z.clone(), dev(path), dev(ua), dev(u)]
    e = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    outs = [[e(b), e(b, B_), e(b), e(b)] for _ in range(2)]
    tok, prob = e(b), torch.empty((b, B_, V), device="cuda")
    call = lambda o, s: B.dflash2_verify_logits(buf[1], None, buf[0], *st, buf[2], buf[3], *o, ws, stream=s)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call(outs[0], None)
    s.synchronize()
    for x, y in zip(want, outs[0]):
        np.testing.assert_array_equal(x, y.cpu().numpy())
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(o, None)
            B.dflash2_sample(buf[0][:, 0], *st, buf[3], tok)
            B.dflash2_target_probs(buf[0], *st, prob)
        graphs.append(g)
    for new, w in (((z2, path2, ua2, u2), want2), ((z, path, ua, u), want)):
        for d, v in zip(buf, new):
            d.copy_(v if torch.is_tensor(v) else dev(v))
        for g, o in zip(graphs, outs):
            for t in o:
                t.fill_(-9)
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip(w, o):
                np.testing.assert_array_equal(x, y.cpu().numpy())
        assert torch.equal(prob, run_probs(B, buf[0], st))


def test_the_same_call_gives_the_same_bits():
    import torch
    B = lib()
    z, _ = logits_of(8, 30011, "normal", 81)
    st = settings_of(8, (1.1, 5000, 0.9, 0.001))
    first = run_probs(B, z[:, None], st)
    for _ in range(5):
        assert torch.equal(first, run_probs(B, z[:, None], st))
