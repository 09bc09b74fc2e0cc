"""The operators on a pool whose offsets pass 32 bits, and on pages of other sizes than a tile's: the same rows in a small
pool give the same bits, and the 64-bit form the values (tolerances as in test_gpu_attend.py)."""

import pytest

torch = pytest.importorskip("torch")

from test_gpu_attend import CACHES, Case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_speculative_decoding_dflash2_gb300 import binding
    binding.lib()
    return binding


def pool(B, cache, pages):
    dtype = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
    k, v = (torch.empty((pages, 16, 8, 128), dtype=dtype, device="cuda") for _ in range(2))
    ke, ve = (None if cache == "bf16" else torch.empty((pages, 16, 8), dtype=torch.uint8, device="cuda") for _ in range(2))
    return B.PagedCache(k, v, ke, ve)


@pytest.mark.parametrize("cache", CACHES)
def test_offsets_past_32_bits(B, cache):
    many = 2 ** 32 // (16 * 8 * 128 * (2 if cache == "bf16" else 1)) + 64
    i32 = dict(dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    k, v, q = (torch.randn((n, h, 128), generator=gen, device="cuda").bfloat16() for n, h in ((190, 8), (190, 8), (4, 32)))
    off, zero = torch.tensor([0, 120, 190], **i32), torch.zeros(2, **i32)
    lens = torch.tensor([120, 70], **i32)
    results = []
    for pages, first in ((16, 0), (many, many - 16)):
        c = pool(B, cache, pages)
        table = (torch.randperm(16, generator=torch.Generator().manual_seed(4)).view(2, 8) + first).to(torch.int32).cuda()
        B.dflash2_cache_append(c, table, zero, k, v, off)
        back = [torch.zeros_like(k), torch.zeros_like(v)]
        B.dflash2_cache_read(c, table, None, off, *back)
        ws = torch.zeros(B.dflash2_attend_workspace(c, 2, 2, 32), dtype=torch.uint8, device="cuda")
        outs = []
        for mode in (1, 2):
            B.dflash2_test_force_attend(mode)
            try:
                out = torch.zeros((2, 2, 32, 128), dtype=torch.bfloat16, device="cuda")
                B.dflash2_attend(c, table, lens, q.view(2, 2, 32, 128), out, ws)
                outs.append(out)
            finally:
                B.dflash2_test_force_attend(0)
        torch.cuda.synchronize()
        assert B.dflash2_read_device_status(ws) == 0
        results.append(back + outs)
        del c
        torch.cuda.empty_cache()
    for small, large in zip(*results):
        assert torch.isfinite(small).all() and torch.equal(small, large)
    if cache == "bf16":
        assert torch.equal(results[1][0], k) and torch.equal(results[1][1], v)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("page", [64, 256, 2048])
@pytest.mark.parametrize("mode", [1, 2])
def test_pages_of_other_sizes(B, cache, page, mode):
    B.dflash2_test_force_attend(mode)
    try:
        Case(B, cache, 128, page, 8, 2, 3, [700, 3, 2048, 2049], seed=30).check()
        Case(B, cache, 128, page, 8, 2, 3, [700, 530, 600], shared=523, seed=31).check(window=300)
    finally:
        B.dflash2_test_force_attend(0)
