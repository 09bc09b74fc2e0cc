"""Pipeline waits of the tcgen05 4-bit contraction that run out (no activations
are copied, and the waits' limit is 1 ms): the kernel ends by itself, its
outputs are NaN, a draft step's status word says so, and the next call on the
same buffers is whole again."""

import numpy as np
import pytest

import dflash2_synth as S
from tests.helpers import Case, lib

pytestmark = pytest.mark.gpu


@pytest.fixture
def give_up():
    B = lib()
    T = B.testing_lib()

    def switch(on):
        assert T.dflash2_test_w4_withhold(int(on)) == 0
    yield switch
    switch(False)


# inputs split over a cluster of up to 8 CTAs, one CTA a tile, several tiles a CTA
@pytest.mark.parametrize("M,K,N", [(300, 4096, 40), (128 * 152, 512, 33), (128 * 400, 256, 100), (1000, 192, 300)])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_a_call_that_gives_up_writes_nan_and_ends(give_up, M, K, N, group, dt):
    import torch
    B = lib()
    codes = torch.randint(0, 256, (M, K // 2), dtype=torch.uint8, device="cuda")
    scale = (torch.rand((M, K // group), device="cuda") * 0.01 + 0.01).to(torch.bfloat16)
    x = torch.randn((N, K), device="cuda").to(torch.bfloat16)
    out = torch.empty((N, M), dtype=getattr(torch, dt), device="cuda")
    B.dflash2_linear_w4(codes, scale, group, x, out)
    want = out.clone()
    assert not torch.isnan(want).any()
    for _ in range(3):
        give_up(True)
        out.zero_()
        B.dflash2_linear_w4(codes, scale, group, x, out)
        torch.cuda.synchronize()
        assert torch.isnan(out).all()
        give_up(False)
        B.dflash2_linear_w4(codes, scale, group, x, out)
        assert torch.equal(out, want)


def test_a_draft_step_that_gives_up_says_so(give_up):
    import torch
    B = lib()
    cfg = S.small_bf16_config(dtype="w4", n_q_heads=8, index=23)
    ctx = [5, 17, 40, 0, 64, 3, 31, 90, 12, 8]
    case = Case(cfg, ctx_lens=ctx, n_new=[1, 2, 8, 3, 0, 5, 1, 4, 2, 6], seed=23).run_gpu()
    assert case.status == 0
    r = case.runner
    want = r.cand_id.clone(), r.cand_logit.clone()
    off = case.dev(np.concatenate([[0], np.cumsum(case.n_new)]).astype(np.int32))
    args = (case.dev(case.ctx_lens), S.to_torch(case.taps_new), off, case.dev(case.anchor))
    give_up(True)
    r.draft(*args)
    torch.cuda.synchronize()
    assert r.device_status() == B.DEV_WAIT_TIMEOUT
    give_up(False)
    r.draft(*args)
    torch.cuda.synchronize()
    assert r.device_status() == 0
    assert torch.equal(r.cand_id, want[0]) and torch.equal(r.cand_logit, want[1])


def test_the_switch_takes_0_and_1(give_up):
    T = lib().testing_lib()
    assert T.dflash2_test_w4_withhold(2) == -1 and T.dflash2_test_w4_withhold(-1) == -1
