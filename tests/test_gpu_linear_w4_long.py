"""The 4-bit product with more inputs than a block's shared memory holds
activations for (9 to 16 rows: above 24576, up to 8 rows: above 49152), which
are then staged window by window, against float64.

Tolerance: every product is exact in fp32.  A sum of K terms is built in steps
of at least 16 terms, each off by at most 2^-22 of the absolute sum S, then K /
group scaled group sums, each step off by at most 2^-23 S: |error| <= S (K / 16
+ K / group + 2) 2^-22.
"""

import pytest

from tests.helpers import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,N", [(24576, 16), (24704, 9), (25600, 16), (49280, 12), (74240, 9),
                                 (49152, 8), (49280, 1), (50176, 8), (99200, 3)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [50, 10500])  # (10500: several row blocks a cluster)
def test_windows_of_activations(K, N, group, M):
    import torch
    B = lib()
    g = torch.Generator(device="cuda")
    g.manual_seed(K + N + M)
    codes = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = (torch.rand((M, K // group), generator=g, device="cuda") * 0.01 + 1e-3).to(torch.bfloat16)
    x = torch.randn((N, K), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full((N, M), float("nan"), device="cuda")
    B.dflash2_linear_w4(codes, scale, group, x, out)
    again = torch.full((N, M), float("nan"), device="cuda")
    B.dflash2_linear_w4(codes, scale, group, x, again)
    assert torch.equal(out, again)
    for lo in range(0, M, 2100):
        c = codes[lo:lo + 2100]
        w = torch.stack((c & 15, c >> 4), 2).reshape(c.shape[0], K).double() - 8
        w = (w.reshape(c.shape[0], K // group, group) * scale[lo:lo + 2100].double()[:, :, None]).reshape(c.shape[0], K)
        want, S = x.double() @ w.t(), x.double().abs() @ w.abs().t()
        assert ((out[:, lo:lo + 2100].double() - want).abs() <= S * (K / 16 + K / group + 2) * 2.0 ** -22).all()


@pytest.mark.parametrize("K,N,group", [(24608, 10, 32), (49248, 2, 32), (49216, 7, 64)])
def test_windows_that_end_inside_a_chunk(K, N, group):
    import torch
    B = lib()
    M = 300
    q = torch.randint(0, 16, (M, K), device="cuda", dtype=torch.uint8)
    scale = torch.ones((M, K // group), dtype=torch.bfloat16, device="cuda")
    x = torch.randint(-8, 9, (N, K), device="cuda").to(torch.bfloat16)
    out = torch.full((N, M), float("nan"), device="cuda")
    B.dflash2_linear_w4(q[:, 0::2] | (q[:, 1::2] << 4), scale, group, x, out)
    # (whole sums below 2^24: exact)
    assert torch.equal(out.double(), x.double() @ (q.double() - 8).t())
