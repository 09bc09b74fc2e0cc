"""dflash2_attend at the largest sizes that it takes: 1024 tokens, 1024 query heads, 256 kv heads, one by one and
together, and values as large as the header allows for.  Tolerances as in test_gpu_attend.py."""

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
@pytest.mark.parametrize("nq,nkv,n_tok,lens,shared", [
    (2, 1, 1024, [1100], 0), (1, 1, 1024, [1024, 700], 0), (1024, 1, 1, [40, 3], 0), (1024, 256, 1, [35], 0),
    (256, 256, 2, [20, 150], 16), (3, 1, 1024, [1090, 1024], 48)])
def test_one_by_one(B, cache, d, nq, nkv, n_tok, lens, shared):
    Case(B, cache, d, 16, nq, nkv, n_tok, lens, shared=shared, seed=70).check()


@pytest.mark.parametrize("cache", CACHES)
def test_all_together(B, cache):
    """One sequence of 1024 tokens of 1024 heads over 256 kv heads; three kv heads of it are compared."""
    gen = torch.Generator(device="cuda").manual_seed(71)
    keys, page, nkv, nq, d, n = 1030, 16, 256, 1024, 128, 1024
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    k, v, q = draw(keys, nkv, d), draw(keys, nkv, d), draw(1, n, nq, d)
    pages = -(-keys // page)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dtype = torch.bfloat16 if cache == "bf16" else torch.uint8
    pool = [torch.zeros((pages, page, nkv, d), dtype=dtype, device="cuda") for _ in range(2)]
    exps = [None, None]
    if cache == "e4m3":
        pool = [x.view(torch.float8_e4m3fn) for x in pool]
        exps = [torch.ones((pages, page, nkv), dtype=torch.uint8, device="cuda") for _ in range(2)]
    c = B.PagedCache(*pool, *exps)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).to(torch.int32).view(1, -1).cuda()
    B.dflash2_cache_append(c, table, i32([0]), k, v, i32([0, keys]))
    back = [torch.zeros_like(k), torch.zeros_like(v)]
    B.dflash2_cache_read(c, table, None, i32([0, keys]), *back)
    ws = torch.zeros(B.dflash2_attend_workspace(c, 1, n, nq), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    B.dflash2_attend(c, table, i32([keys]), q, out, ws)
    torch.cuda.synchronize()
    assert B.dflash2_read_device_status(ws) == 0
    hidden = torch.arange(keys, device="cuda") >= (keys - n + 1 + torch.arange(n, device="cuda"))[:, None]
    for h in (0, 100, 255):
        z = torch.einsum("tgd,kd->gtk", q[0, :, 4 * h:4 * h + 4].double(), back[0][:, h].double()) * d ** -0.5
        p = torch.softmax(z.masked_fill(hidden, float("-inf")), -1)
        want, mag = (torch.einsum("gtk,kd->tgd", p, x) for x in (back[1][:, h].double(), back[1][:, h].double().abs()))
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -9 + 2.0 ** -16 if cache == "e4m3" else 2.0 ** -14) * mag
        assert ((out[0, :, 4 * h:4 * h + 4].double() - want).abs() <= tol).all(), h


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("step", [1, -1])
def test_values_near_the_largest_that_many_keys_allow(B, cache, step):
    """Values up to 2^102 under 400 keys (|value| times keys below 2^111), with scores that rise or fall by 60."""
    n = 400
    c = Case(B, cache, 128, 16, 2, 1, 3, [n, 17], seed=72, spread=0.0)
    for i, keys in enumerate(c.lens):
        for p in range(keys):
            page = int(c.table[i, p // 16])
            c.pool["v"][page, p % 16] = 2.0 ** 102 * (1 if p % 3 else -1)
            c.pool["k"][page, p % 16] = 0
            c.pool["k"][page, p % 16, :, 0] = step * (60.0 * p / n - 30.0)
    c.q[:] = 0
    c.q[..., 0] = 11.3125
    c.quantise()
    c.check()
