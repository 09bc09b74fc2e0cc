"""The product with 4-bit weights and group scales (dflash2_linear_w4)
against the same product in float64.

Tolerance: every product of a whole number in -8..7 and a bf16 value is exact
in fp32.  A sum of K terms is built in steps of at least 16 terms, each step
off by at most 2^-22 of the absolute sum S = sum |scale q x| (a matrix unit
may truncate instead of rounding, and its terms are aligned to the largest),
then K / group scaled group sums, each step off by at most 2^-23 S: |error| <=
S (K / 16 + K / group + 2) 2^-22.  A bf16 output adds half a step, 2^-8 of its
value (2^-8 of the sum with the old value when accumulating).
"""

import numpy as np
import pytest

from tests.helpers import lib

pytestmark = pytest.mark.gpu


def weights(M, K, group, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = torch.randint(0, 16, (M, K), generator=g, device="cuda", dtype=torch.uint8)
    scale = (torch.rand((M, K // group), generator=g, device="cuda") * 0.01 + 1e-3).to(torch.bfloat16)
    return q[:, 0::2] | (q[:, 1::2] << 4), q, scale


def reference(q, scale, group, x):
    """(product, absolute sums) in float64."""
    w = (q.double() - 8) * scale.double().repeat_interleave(group, 1)
    return x.double() @ w.t(), x.double().abs() @ w.abs().t()


def check(got, want, S, K, group, old=None):
    import torch
    tol = S * (K / 16 + K / group + 2) * 2.0 ** -22
    total = want if old is None else want + old.double()
    if old is not None:
        tol = tol + total.abs() * 2.0 ** -24
    if got.dtype == torch.bfloat16:
        tol = tol + (total.abs() + tol) * 2.0 ** -8
    bad = (got.double() - total).abs() > tol
    assert not bad.any(), (int(bad.sum()), (got.double() - total).abs().max().item())


def case(M, K, N, group, seed=0):
    import torch
    codes, q, scale = weights(M, K, group, seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    x = torch.randn((N, K), generator=g, device="cuda").to(torch.bfloat16)
    return codes, q, scale, x


@pytest.mark.parametrize("M,K", [(1, 128), (7, 256), (16, 128), (17, 384), (128, 1024), (1000, 640), (2051, 4096),
                                 (300, 12288), (33, 17408)])
@pytest.mark.parametrize("N", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 130, 257])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_against_float64(M, K, N, group):
    import torch
    B = lib()
    codes, q, scale, x = case(M, K, N, group, seed=M + N)
    want, S = reference(q, scale, group, x)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((N, M), float("nan"), dtype=dt, device="cuda")
        B.dflash2_linear_w4(codes, scale, group, x, out)
        check(out, want, S, K, group)


@pytest.mark.parametrize("K,group", [(32, 32), (64, 32), (96, 32), (64, 64), (192, 64), (320, 64), (2688, 64),
                                     (128, 128), (2688, 128), (8064, 128), (160, 32)])
@pytest.mark.parametrize("N", [1, 5, 40, 100])
def test_short_and_odd_inner_sizes(K, group, N):
    import torch
    B = lib()
    codes, q, scale, x = case(77, K, N, group, seed=K)
    want, S = reference(q, scale, group, x)
    out = torch.full((N, 77), float("nan"), device="cuda")
    B.dflash2_linear_w4(codes, scale, group, x, out)
    check(out, want, S, K, group)


@pytest.mark.parametrize("N", [1, 8, 50, 200])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strided_rows_accumulate_and_untouched_surroundings(N, dt):
    """x and out as columns of wider buffers; what lies beside out stays, what
    lies beside x is NaN."""
    import torch
    B = lib()
    M, K, group = 203, 512, 64
    codes, q, scale, x0 = case(M, K, N, group, seed=3)
    xb = torch.full((N, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = xb[:, 16:16 + K]
    x.copy_(x0)
    want, S = reference(q, scale, group, x0)
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    ob = torch.randn((N + 1, M + 5), device="cuda").to(dtype)
    keep = ob.clone()
    out = ob[:N, 3:3 + M]
    old = out.clone()
    B.dflash2_linear_w4(codes, scale, group, x, out, accumulate=True)
    check(out, want, S, K, group, old)
    B.dflash2_linear_w4(codes, scale, group, x, out)
    check(out, want, S, K, group)
    out.copy_(keep[:N, 3:3 + M])
    assert torch.equal(ob, keep)


def test_extreme_codes_scales_and_inputs():
    import torch
    B = lib()
    M, K, group = 64, 256, 32
    for c in (0, 8, 15):
        q = torch.full((M, K), c, dtype=torch.uint8, device="cuda")
        codes = q[:, 0::2] | (q[:, 1::2] << 4)
        scale = torch.ones((M, K // group), dtype=torch.bfloat16, device="cuda")
        x = torch.ones((3, K), dtype=torch.bfloat16, device="cuda")
        out = torch.empty((3, M), device="cuda")
        B.dflash2_linear_w4(codes, scale, group, x, out)
        assert torch.equal(out, torch.full_like(out, float((c - 8) * K)))  # whole numbers: exact
    codes, q, scale, x = case(M, K, 4, group, seed=9)
    scale[5], scale[6, 0] = 0.0, float("inf")
    x[1, 7], x[2, 100] = float("nan"), float("inf")
    out = torch.empty((4, M), device="cuda")
    B.dflash2_linear_w4(codes, scale, group, x, out)
    rest = [m for m in range(M) if m not in (5, 6)]
    want, S = reference(q, scale, group, x)
    check(out[[0, 3]][:, rest], want[[0, 3]][:, rest], S[[0, 3]][:, rest], K, group)
    assert torch.isnan(out[1]).all()            # a NaN input reaches every output of its row only
    assert not torch.isfinite(out[2][q[:, 100] != 8]).any()
    assert (out[[0, 3], 5] == 0).all() and not torch.isfinite(out[[0, 3], 6]).any()


def test_no_rows_and_large_row_counts():
    import torch
    B = lib()
    codes, q, scale, x = case(40, 128, 70000, 128, seed=4)
    out = torch.full((70000, 40), float("nan"), device="cuda")
    B.dflash2_linear_w4(codes, scale, 128, x, out)
    want, S = reference(q, scale, 128, x)
    check(out, want, S, 128, 128)
    keep = out.clone()
    B.dflash2_linear_w4(codes, scale, 128, x[:0], out[:0])
    assert torch.equal(out, keep)


def test_offsets_past_32_bits():
    """Rows whose codes, inputs and outputs start beyond 2^32 bytes."""
    import torch
    B = lib()
    M, K, group = 2_200_000, 4096, 128
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device="cuda")
    scale = torch.ones((M, K // group), dtype=torch.bfloat16, device="cuda")
    tail, q, st, x = case(300, K, 2, group, seed=6)
    codes[-300:], scale[-300:] = tail, st
    codes[:-300] = 0x99                       # weight 1 everywhere else
    buf = torch.zeros((2, (1 << 31) + 8), dtype=torch.bfloat16, device="cuda")
    xw = buf[:, :K]
    xw.copy_(x)
    out = torch.empty((2, M), device="cuda")
    B.dflash2_linear_w4(codes, scale, group, xw, out)
    want, S = reference(q, st, group, x)
    check(out[:, -300:], want, S, K, group)
    ones = x.double().sum(1, keepdim=True)
    assert ((out[:, :-300].double() - ones).abs() <= x.double().abs().sum(1, keepdim=True) * 300 * 2.0 ** -22).all()


def test_other_stream_graph_and_repeats():
    import torch
    B = lib()
    M, K, N, group = 777, 2048, 8, 64
    codes, q, scale, x = case(M, K, N, group, seed=11)
    out = torch.empty((N, M), device="cuda")
    B.dflash2_linear_w4(codes, scale, group, x, out)
    first = out.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(3):
            out.fill_(float("nan"))
            B.dflash2_linear_w4(codes, scale, group, x, out)
    s.synchronize()
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        B.dflash2_linear_w4(codes, scale, group, x, out)
    x2 = torch.randn((N, K), device="cuda").to(torch.bfloat16)
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    want, S = reference(q, scale, group, x2)
    check(out, want, S, K, group)


def test_rows_do_not_depend_on_their_neighbours():
    """A row's output is the same bits alone and in a batch of its size class."""
    import torch
    B = lib()
    codes, q, scale, x = case(500, 1024, 8, 64, seed=21)
    out = torch.empty((8, 500), device="cuda")
    B.dflash2_linear_w4(codes, scale, 64, x, out)
    y = x.clone()
    y[[0, 1, 2, 4, 5, 6, 7]] = 7.0
    out2 = torch.empty_like(out)
    B.dflash2_linear_w4(codes, scale, 64, y, out2)
    assert torch.equal(out[3], out2[3])
