"""DraftRunner as a server drives it with request settings: draft, select, the target's logits changed by adjust_logits
for the selected path, verify_logits on them, in place and into a buffer of their own."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import operator_reference as OR  # noqa: E402
import sampling_reference as SR  # noqa: E402
import dflash2_synth as S  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
def test_a_step_with_settings(in_place):
    from block_speculative_decoding_dflash2_gb300 import binding as B
    from block_speculative_decoding_dflash2_gb300.runner import DraftRunner
    cfg = S.small_bf16_config(batch=2)
    rng = np.random.default_rng(80)
    batch, rows, vocab, ctx = 2, cfg["block_size"], cfg["vocab"], 40
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda")  # noqa: E731
    r = DraftRunner(cfg, S.device_weights(S.make_weights(cfg)), batch, ctx + 16, max_new=batch * ctx)
    taps = S.to_torch(S.make_taps(cfg, batch * ctx, stream="settings"))
    r.append(i32([0, 0]), taps, i32([0, ctx, 2 * ctx]))
    anchor = i32([17, 5])
    r.draft(i32([ctx, ctx]), None, i32([0, 0, 0]), anchor)
    r.select(anchor)
    path = r.path.cpu().numpy()
    logits = f32(rng.standard_normal((batch, rows, vocab)) * 3)
    z = logits.double().cpu().numpy()
    tokens, n, prompt = rng.integers(0, vocab, (batch, 60)), [60, 25], [20, 30]
    rho, presence, frequency = [1.3, 1.0], [0.4, 0.0], [0.2, 0.0]
    # the first draft of each sequence is liked by a bias
    bias_id, bias = [[path[0, 0], 3], [path[1, 0], -1]], [[40.0, -2.0], [40.0, 0.0]]
    words = -(-vocab // 32)
    mask = rng.integers(-2 ** 31, 2 ** 31, (batch, rows, words), dtype=np.int64).astype(np.int32)
    mask[1] = -1
    mask[0, 0, path[0, 0] // 32] |= np.array(1 << (path[0, 0] % 32), np.uint32).astype(np.int32)
    out = logits if in_place else torch.zeros_like(logits)
    r.adjust_logits(logits, i32(tokens), i32(n), None if in_place else out, i32(prompt), f32(rho), f32(presence),
                    f32(frequency), i32(bias_id), f32(bias), i32(mask))
    ua, u = f32(rng.random((batch, rows - 1)) * 0.5), f32(rng.random(batch))
    r.verify_logits(out, ua, u, temperature=f32([0.8, 0.0]))
    torch.cuda.synchronize()
    assert r.device_status() == 0 and B.dflash2_read_device_status(r.verify_ws) == 0
    if not in_place:
        assert np.array_equal(logits.double().cpu().numpy(), z)
    got = out.double().cpu().numpy()
    accepted = 0
    for s in range(batch):
        bits = np.unpackbits(mask[s].view(np.uint8).reshape(rows, -1), axis=1, bitorder="little")
        for i in range(rows):
            want = OR.adjust(z[s, i], tokens[s, :n[s]].tolist(), prompt[s], path[s, :i].tolist(), float(np.float32(rho[s])),
                             float(np.float32(presence[s])), float(np.float32(frequency[s])),
                             [(t, b) for t, b in zip(bias_id[s], bias[s]) if t >= 0], bits[i])
            gone = np.isneginf(want)
            assert np.array_equal(np.isneginf(got[s, i]), gone)
            # six fp32 steps, none above the sum of the terms' magnitudes
            assert np.abs(got[s, i][~gone] - want[~gone]).max() <= 6 * 2.0 ** -24 * (2 * np.abs(z[s, i]).max() + 60)
        spec = (float(np.float32(0.8)) if s == 0 else 0.0, 0, 1.0, 0.0)
        a, tok = SR.verify(got[s], path[s], rows - 1, spec, ua[s].cpu().numpy(), float(u[s]))
        assert (int(r.accept_len[s]), int(r.next_anchor[s])) == (a, tok)
        accepted += a
    assert accepted > 0
