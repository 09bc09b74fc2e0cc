"""Draws and top-p borders on rows where most of the mass lies in many equal or
nearly equal small tokens, so that errors of single masses add up, against
float64.

Masses are good to 2^-35 of themselves and a unit, which at these sizes is at
most 2^-55 of the row's mass (2^18 tokens: 2^-37 of it together), so a running
sum and a share of the total are within 2^-34 of the total each: draws and
borders whose threshold is within 2^-33 of a running sum are left out (one in
10^4 or less), all others are compared exactly.
"""

import numpy as np
import pytest

from tests.helpers import lib

pytestmark = pytest.mark.gpu

NEAR = 2.0 ** -33


def row_of(kind, depth, V, g):
    z = np.full(V, -depth, np.float32)
    if kind == "two values":
        z[::2] -= np.float32(0.21)
    elif kind == "random":
        z += g.standard_normal(V).astype(np.float32)
    z[V // 3] = 0.0
    return z


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("kind", ["equal", "two values", "random"])
@pytest.mark.parametrize("depth", [5, 8, 10, 11, 12, 13, 14, 16, 18, 21])
@pytest.mark.parametrize("V", [50257, 151936])
def test_draws_from_small_tokens(V, depth, kind, dtype):
    import torch
    B = lib()
    g = np.random.default_rng(depth)
    n = 4000
    z = torch.from_numpy(row_of(kind, depth, V, g)).cuda().to(getattr(torch, dtype))
    temp = torch.full((n,), 1.0, device="cuda")
    u = torch.from_numpy(g.random(n, dtype=np.float32)).cuda()
    tok = torch.empty((n,), dtype=torch.int32, device="cuda")
    for lo in range(0, n, 200):  # (rows at a stride of zero are refused)
        B.dflash2_sample(z.expand(200, V).contiguous(), temp[:200], None, None, None, u[lo:lo + 200], tok[lo:lo + 200])
    c = (z.double() - z.double().max()).exp().cumsum(0)
    t = u.double() * c[-1]
    want = torch.searchsorted(c, t, right=True)
    border = torch.minimum((c[want] - t).abs(), (t - torch.where(want > 0, c[(want - 1).clamp(min=0)], 0.0)).abs())
    clear = border > NEAR * c[-1]
    assert clear.double().mean() > 1 - 1e-3
    assert torch.equal(tok[clear].long(), want[clear])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("kind", ["equal", "two values", "random"])
@pytest.mark.parametrize("depth", [5, 10, 12, 13, 14, 16])
def test_top_p_borders_among_small_tokens(depth, kind, dtype):
    import torch
    B = lib()
    V, n = 151936, 64
    g = np.random.default_rng(100 + depth)
    z = torch.from_numpy(row_of(kind, depth, V, g)).cuda().to(getattr(torch, dtype))
    top_p = torch.from_numpy(g.uniform(0.5, 0.9999, n).astype(np.float32)).cuda()
    prob = torch.empty((n, 1, V), device="cuda")
    B.dflash2_target_probs(z.expand(n, 1, V).contiguous(), None, None, top_p, None, prob)
    zs, ids = torch.sort(z.float(), descending=True, stable=True)
    c = (zs.double() - zs[0].double()).exp().cumsum(0)
    t = top_p.double() * c[-1]
    last = torch.searchsorted(c, t)  # the first running mass of at least t
    clear = torch.minimum((c[last] - t).abs(), (t - torch.where(last > 0, c[(last - 1).clamp(min=0)], 0.0)).abs()) > NEAR * c[-1]
    assert clear.double().mean() > 0.9
    kept = (prob[:, 0] > 0).sum(1)
    assert torch.equal(kept[clear], last[clear] + 1)
    for r in (0, n // 2, n - 1):
        if clear[r]:
            assert (prob[r, 0][ids[:int(last[r]) + 1]] > 0).all()


def test_acceptance_of_small_tokens():
    """The draft's token holds a 2^-18th of a row of equal tokens below one
    larger one: accepted up to its probability in float64, to 2^-20 of it."""
    import torch
    B = lib()
    V, depth = 151936, 13
    z = np.full(V, -depth, np.float32)
    z[7] = 0.0
    p = np.exp(-float(depth)) / (1 + (V - 1) * np.exp(-float(depth)))
    ua = np.float32(p) * np.array([1 - 2.0 ** -20, 1 - 2.0 ** -22, 1 + 2.0 ** -22, 1 + 2.0 ** -20], np.float64)
    ua = ua.astype(np.float32)
    b = len(ua)
    zt = torch.from_numpy(np.broadcast_to(z, (b, 2, V)).copy()).cuda()
    i32 = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")
    acc, out, n, nxt = i32(b), i32(b, 2), i32(b), i32(b)
    path = torch.full((b, 1), 1000, dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.dflash2_verify_logits_workspace(b, 2), dtype=torch.uint8, device="cuda")
    B.dflash2_verify_logits(path, None, zt, None, None, None, None, torch.from_numpy(ua[:, None]).cuda(),
                            torch.full((b,), 0.5, device="cuda"), acc, out, n, nxt, ws)
    assert acc.tolist() == [int(float(x) < p) for x in ua]
