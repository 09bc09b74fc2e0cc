"""The 4-bit-weight path (DFLASH2_W4: codes with bf16 group scales, bf16
activations): draft-step parity with the oracle on the dequantised weights,
stage by stage and end to end, the selector on its per-step and table paths,
and a speculative step whose target shares the 4-bit lm_head."""

import numpy as np
import pytest

import dflash2_synth as S
import oracle as O
from tests import sampling_reference as R
from tests.helpers import Case, lib
from tests.test_gpu_draft import check_case
from tests.test_gpu_full_configs import check_select_and_verify
from tests.test_gpu_stagewise import run_stagewise

pytestmark = pytest.mark.gpu

TOL = 2e-2  # the bf16 workloads' bound on a logit


def small_w4(**over):
    return S.small_bf16_config(dtype="w4", **over)


def test_w4_small_one_layer_stagewise():
    cfg = small_w4(n_layers=1, index=21)
    case = Case(cfg, ctx_lens=[60, 0, 150], n_new=[3, 8, 1], seed=21).run_gpu()
    assert case.status == 0
    run_stagewise(case)
    check_case(case, TOL)


def test_w4_small_two_layers_ragged_batch():
    cfg = small_w4(index=22)
    case = Case(cfg, ctx_lens=[40, 0, 200], n_new=[1, 8, 3], seed=22).run_gpu()
    check_case(case, TOL)
    check_select_and_verify(case, [0, 1, 2], None, "w4 small, two layers")


def test_w4_small_wide_batch():
    # 10 sequences of 8 rows: the contractions for many rows
    cfg = small_w4(n_q_heads=8, index=23)
    ctx = [5, 17, 40, 0, 64, 3, 31, 90, 12, 8]
    case = Case(cfg, ctx_lens=ctx, n_new=[1, 2, 8, 3, 0, 5, 1, 4, 2, 6], seed=23).run_gpu()
    check_case(case, TOL)


def test_w4_without_convolution_or_new_rows():
    cfg = small_w4(index=25, conv_kernel_size=0)
    check_case(Case(cfg, ctx_lens=[33, 9], n_new=[0, 0], seed=25).run_gpu(), TOL)


def test_w4_select_paths_agree():
    cfg = small_w4(index=24)
    case = Case(cfg, ctx_lens=[30, 77], n_new=[4, 4], seed=24).run_gpu()
    assert case.status == 0
    r = case.runner
    anchor = case.dev(case.anchor)
    r.select(anchor)
    p_gemm = r.path.cpu().numpy().copy()
    r.build_selector_table()
    r.select(anchor)
    p_table = r.path.cpu().numpy()
    cid, cz = r.cand_id.cpu().numpy(), r.cand_logit.cpu().numpy().astype(np.float64)
    for s in range(case.b):
        p, _, _ = O.select_path(cfg, case.Wv, int(case.anchor[s]), cid[s], cz[s])
        assert list(p_gemm[s]) == list(p) and list(p_table[s]) == list(p)


def test_w4_draft_step_in_a_captured_graph():
    """Two replays on one workspace give the eager step's logits."""
    import torch
    cfg = small_w4(index=26)
    case = Case(cfg, ctx_lens=[40, 100], n_new=[2, 5], seed=26).run_gpu()
    want = case.runner.cand_logit.clone()
    r = case.runner
    off = case.dev(np.concatenate([[0], np.cumsum(case.n_new)]).astype(np.int32))
    args = (case.dev(case.ctx_lens), S.to_torch(case.taps_new), off, case.dev(case.anchor))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.draft(*args)
    for _ in range(2):
        r.cand_logit.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.cand_logit, want)
    assert r.device_status() == 0


def test_w4_config_checks():
    B = lib()
    assert B.dflash2_validate_config(B.make_config(small_w4())) == 0
    assert B.dflash2_validate_config(B.make_config(small_w4(hidden=288))) == -2      # not whole groups
    assert B.dflash2_validate_config(B.make_config(small_w4(intermediate=672))) == -2
    for name in ("qwen3_8b_b1", "qwen3_27b_b8", "a3b_30b_fp8"):
        assert B.dflash2_validate_config(B.make_config(S.config_of(name, dtype="w4"))) == 0
    cfg = small_w4()
    W = S.device_weights(S.make_weights(cfg))
    c, ws = B.make_config(cfg), None
    import torch
    w = B.WeightSet(W)
    ids = torch.zeros((1, 7, 8), dtype=torch.int32, device="cuda")
    z = torch.zeros((1, 7, 8), device="cuda")
    path = torch.zeros((1, 7), dtype=torch.int32, device="cuda")
    with pytest.raises(B.DFlash2Error) as e:
        B.dflash2_select_path_static(c, w, 1, ids[0, 0, :1].contiguous(), ids, z, path, None)
    assert e.value.status == -7
    del W["scales"]
    nows = torch.zeros(B.dflash2_workspace_size(c, 1, 0, 16), dtype=torch.uint8, device="cuda")
    with pytest.raises(B.DFlash2Error) as e:
        B.dflash2_select_path(c, B.WeightSet(W), 1, ids[0, 0, :1].contiguous(), ids, z, path, None, nows)
    assert e.value.status == -1


def test_speculative_steps_with_the_shared_4bit_lm_head():
    """Draft with 4-bit weights, select, the target's logits of the verify
    batch as the 4-bit lm_head's product with its (given) hidden states,
    sampled verification from those logits, and the first anchor sampled the
    same way; each step's tokens against the float64 definition on the
    product's own logits, the product against float64."""
    import torch
    B = lib()
    cfg = small_w4(index=27)
    b, B_, V, H = 3, cfg["block_size"], cfg["vocab"], cfg["hidden"]
    case = Case(cfg, ctx_lens=[20, 0, 75], n_new=[4, 2, 6], seed=27)
    r = case.runner
    lm = r.w.tensors["lm_head"], r.w.tensors["scales"]["lm_head"]
    lm_v = case.W["lm_head"].values
    g = np.random.default_rng(5)
    hidden = lambda n: torch.from_numpy(g.standard_normal((n, H)).astype(np.float32)).cuda().to(torch.bfloat16)
    f32 = lambda *s: torch.from_numpy(g.random(s, dtype=np.float32)).cuda()
    full = lambda v, t: torch.full((b,), v, dtype=t, device="cuda")
    settings = full(8.0, torch.float32), full(50, torch.int32), full(0.9, torch.float32), None
    spec = (8.0, 50, float(np.float32(0.9)), 0.0)

    def logits_of(h):
        out = torch.empty((h.shape[0], V), device="cuda")
        B.dflash2_linear_w4(*lm, B.W4_GROUP, h, out)
        want = h.double().cpu().numpy() @ lm_v.T
        S_ = np.abs(h.double().cpu().numpy()) @ np.abs(lm_v).T
        assert np.all(np.abs(out.cpu().numpy() - want) <= S_ * (H / 16 + H / 64 + 2) * 2.0 ** -22)
        return out

    # the first anchor of every sequence
    z = logits_of(hidden(b))
    anchor = torch.empty((b,), dtype=torch.int32, device="cuda")
    u = f32(b)
    B.dflash2_sample(z, *settings, u, anchor)
    zv, uv = z.double().cpu().numpy(), u.cpu().numpy()
    assert list(anchor.cpu().numpy()) == [R.draw(R.masses(zv[s], *spec), uv[s]) for s in range(b)]
    case.anchor = anchor.cpu().numpy()
    case.run_gpu()
    assert case.status == 0
    ctx = case.dev(case.ctx_lens + case.n_new)   # (the toy target gives no taps to append)
    seq = ctx.clone()
    total = 0
    for _ in range(4):
        r.select(anchor)
        z = logits_of(hidden(b * B_)).view(b, B_, V)
        # a target that likes half of the drafts
        path = r.path.cpu().numpy()
        for s in range(b):
            for i in range(B_ - 1):
                if g.random() < 0.5:
                    z[s, i, int(path[s, i])] += 40.0
        ua, us = f32(b, B_ - 1), f32(b)
        r.verify_logits(z, ua, us, *settings, seq_len=seq)
        zv, uav, usv = z.double().cpu().numpy(), ua.cpu().numpy(), us.cpu().numpy()
        for s in range(b):
            a, tok = R.verify(zv[s], path[s], B_ - 1, spec, uav[s], usv[s])
            assert (int(r.accept_len[s]), int(r.next_anchor[s])) == (a, tok)
            assert list(r.out_tok[s].cpu().numpy()) == list(path[s, :a]) + [tok] + [-1] * (B_ - 1 - a)
            total += a
        anchor = r.next_anchor.clone()
        r.draft(ctx, None, torch.zeros((b + 1,), dtype=torch.int32, device="cuda"), anchor)
    assert total > 0 and int(r.counters[2]) == total and int(r.counters[0]) == 4 * b
    assert B.dflash2_read_device_status(r.verify_ws) == 0 and r.device_status() == 0
    assert int(seq.sum()) == int(ctx.sum()) + total + 4 * b
