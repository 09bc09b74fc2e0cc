"""The operators around a target's verification pass, run together as a server would: the drafted block's keys and values
written into an 8-bit cache behind a shared prompt, attention over it, the 4-bit readout, the requests' settings on the
logits, sampled verification.  Several steps, captured in one graph and replayed; each stage against its 64-bit
definition on what the stage before has left."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import operator_reference as OR  # noqa: E402
import sampling_reference as SR  # noqa: E402
import dflash2_synth as S  # noqa: E402

pytestmark = pytest.mark.gpu


def test_steps_of_a_target_with_an_8bit_cache():
    from block_speculative_decoding_dflash2_gb300 import binding as B
    B.lib()
    rng = np.random.default_rng(12)
    b, n_tok, nq, nkv, d, vocab, page, shared = 3, 5, 8, 2, 128, 1000, 16, 48
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(torch.bfloat16)  # noqa: E731
    # pages: three shared ones, eight of its own for each sequence
    order = rng.permutation(3 + 8 * b)
    table = np.concatenate([np.tile(order[:3], (b, 1)), order[3:].reshape(b, 8)], 1).astype(np.int32)
    pool = lambda dt: torch.zeros((order.size, page, nkv, d), dtype=torch.uint8, device="cuda").view(dt)  # noqa: E731
    exps = lambda: torch.ones((order.size, page, nkv), dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = B.PagedCache(pool(torch.float8_e4m3fn), pool(torch.float8_e4m3fn), exps(), exps())
    tab = torch.from_numpy(table).cuda()
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    # the shared prompt once, through the first sequence, then each sequence's own
    own = [7, 20, 1]
    B.dflash2_cache_append(cache, tab[:1].contiguous(), i32([0]), draw(shared, nkv, d), draw(shared, nkv, d), i32([0, shared]), status)
    off = np.concatenate(([0], np.cumsum(own)))
    B.dflash2_cache_append(cache, tab, i32([shared] * b), draw(off[-1], nkv, d), draw(off[-1], nkv, d), i32(off.tolist()), status)
    # what a step reads and writes
    seq_len = i32([shared + n for n in own])  # positions committed
    k, v, q = (torch.zeros((b * n_tok, h, d), dtype=torch.bfloat16, device="cuda") for h in (nkv, nkv, nq))
    new_off, kv_len = i32([n_tok * i for i in range(b + 1)]), torch.zeros((b,), dtype=torch.int32, device="cuda")
    attn = torch.zeros((b, n_tok, nq, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(B.dflash2_attend_workspace(cache, b, n_tok, nq, shared), dtype=torch.uint8, device="cuda")
    lm = S.quantize_groups_w4(rng.standard_normal((vocab, nq * d)).astype(np.float32) * 0.05)
    codes = torch.from_numpy(lm.q).cuda()
    scale = torch.from_numpy(lm.scale.astype(np.float32)).cuda().to(torch.bfloat16)
    logits = torch.zeros((b, n_tok, vocab), device="cuda")
    changed = torch.zeros_like(logits)
    tokens, n_tokens = i32(rng.integers(0, vocab, (b, 200)).tolist()), i32([30, 64, 100])
    path = torch.zeros((b, n_tok - 1), dtype=torch.int32, device="cuda")
    rho, pres, freq = f32([1.2, 1.0, 0.9]), f32([0.5, 0.0, 0.3]), f32([0.1, 0.0, 0.2])
    mask = torch.zeros((b, n_tok, 32), dtype=torch.int32, device="cuda")
    bias_id, bias = i32([[5, 9], [-1, 900], [44, 44]]), f32([[2.0, -3.0], [0.0, 4.0], [1.0, 6.0]])
    settings = f32([1.0, 0.7, 0.0]), i32([50, 0, 0]), f32([0.9, 1.0, 1.0]), None
    ua, u = torch.zeros((b, n_tok - 1), device="cuda"), torch.zeros((b,), device="cuda")
    acc, n_out, nxt = (torch.zeros((b,), dtype=torch.int32, device="cuda") for _ in range(3))
    out_tok = torch.zeros((b, n_tok), dtype=torch.int32, device="cuda")
    vws = torch.zeros(B.dflash2_verify_logits_workspace(b, n_tok), dtype=torch.uint8, device="cuda")

    def step():
        B.dflash2_cache_append(cache, tab, seq_len, k, v, new_off, status)
        torch.add(seq_len, n_tok, out=kv_len)
        B.dflash2_attend(cache, tab, kv_len, q.view(b, n_tok, nq, d), attn, ws, shared_len=shared)
        B.dflash2_linear_w4(codes, scale, 64, attn.view(b * n_tok, nq * d), logits.view(b * n_tok, vocab))
        B.dflash2_adjust_logits(logits, tokens, n_tokens, changed, path=path, repetition=rho, presence=pres, frequency=freq,
                                bias_id=bias_id, bias=bias, mask=mask, workspace=status)
        B.dflash2_verify_logits(path, None, changed, *settings, ua, u, acc, out_tok, n_out, nxt, vws, seq_len=seq_len)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    everything = torch.full((b, n_tok, 32), -1, dtype=torch.int32, device="cuda")
    emitted = 0
    for _ in range(4):
        for t in (k, v, q):
            t.copy_(draw(*t.shape))
        path.copy_(i32(rng.integers(0, vocab, (b, n_tok - 1)).tolist()))
        mask.copy_(everything)
        mask[1] = i32(rng.integers(-2 ** 31, 2 ** 31, (n_tok, 32)).tolist())
        # drafts that the targets like: their biases say so
        path[0, 0], path[1, 0], path[2, 0] = 5, 900, 44
        ua.copy_(f32(rng.random((b, n_tok - 1)).tolist()))
        u.copy_(f32(rng.random(b).tolist()))
        before = seq_len.cpu().numpy().copy()
        graph.replay()
        torch.cuda.synchronize()
        assert B.dflash2_read_device_status(status) == 0 and B.dflash2_read_device_status(ws) == 0
        # attention, on what the cache reads back as
        keys = before + n_tok
        at = np.concatenate(([0], np.cumsum(keys)))
        kk, vv = (torch.zeros((int(at[-1]), nkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        B.dflash2_cache_read(cache, tab, None, i32(at.tolist()), kk, vv)
        kk, vv = kk.double().cpu().numpy(), vv.double().cpu().numpy()
        qq, got = q.view(b, n_tok, nq, d).double().cpu().numpy(), attn.double().cpu().numpy()
        for s in range(b):
            new = k[s * n_tok:(s + 1) * n_tok].double().cpu().numpy()  # (each row's code: half an e4m3 step, or of a subnormal)
            room = 2.0 ** -4 * np.abs(new) + 2.0 ** -10 / 448 * 2 * np.abs(new).max(-1, keepdims=True)
            assert (np.abs(kk[at[s + 1] - n_tok:at[s + 1]] - new) <= room).all()
            want, mag = OR.attend(qq[s], kk[at[s]:at[s + 1]], vv[at[s]:at[s + 1]], d ** -0.5, True, 0)
            assert (np.abs(got[s] - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -16) * mag).all()
        # readout
        x = attn.view(b * n_tok, -1).double().cpu().numpy()
        z, size = x @ lm.values.T, np.abs(x) @ np.abs(lm.values).T
        assert (np.abs(logits.view(b * n_tok, -1).cpu().numpy() - z) <= size * (nq * d / 16 + nq * d / 64 + 2) * 2.0 ** -22).all()
        # settings and verification
        zz, host = logits.double().cpu().numpy(), {n: t.cpu().numpy() for n, t in dict(
            tokens=tokens, n=n_tokens, path=path, rho=rho, pres=pres, freq=freq, bid=bias_id, bias=bias, mask=mask,
            ua=ua, u=u, acc=acc, nxt=nxt, out=out_tok).items()}
        final = changed.double().cpu().numpy()
        for s in range(b):
            bits = np.unpackbits(host["mask"][s].view(np.uint8).reshape(n_tok, -1), axis=1, bitorder="little")
            for i in range(n_tok):
                want = OR.adjust(zz[s, i], host["tokens"][s, :host["n"][s]].tolist(), 0, host["path"][s, :i].tolist(),
                                 float(host["rho"][s]), float(host["pres"][s]), float(host["freq"][s]),
                                 list(zip(host["bid"][s].tolist(), host["bias"][s].tolist())), bits[i])
                gone = np.isneginf(want)
                assert np.array_equal(np.isneginf(final[s, i]), gone)
                assert np.abs(final[s, i][~gone] - want[~gone]).max() <= 6 * 2.0 ** -24 * (2 * np.abs(zz[s, i]).max() + 40)
            spec = tuple(0.0 if t is None else float(t[s]) for t in settings)
            a, tok = SR.verify(final[s], host["path"][s], n_tok - 1, (spec[0], int(spec[1]), spec[2], spec[3]), host["ua"][s],
                               host["u"][s])
            assert (int(host["acc"][s]), int(host["nxt"][s])) == (a, tok)
            assert int(seq_len[s]) == before[s] + a + 1
            emitted += a
    assert emitted > 0
