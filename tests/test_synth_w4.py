"""The 4-bit weight format the W4 workloads are drawn in (input generation,
shared by the oracle and the GPU path): packing, scales, rounding and the
error bound of a group quantisation."""

import numpy as np

import dflash2_synth as S


def unpack(q):
    return np.stack([q & 15, q >> 4], axis=2).reshape(q.shape[0], -1).astype(np.int64) - 8


def test_values_are_the_packed_codes_times_their_scales():
    w = S._rng(1, "w4").standard_normal((7, 256)).astype(np.float32)
    t = S.quantize_groups_w4(w)
    assert t.q.dtype == np.uint8 and t.q.shape == (7, 128) and t.scale.shape == (7, 4)
    v = unpack(t.q) * np.repeat(t.scale.astype(np.float64), 64, axis=1)
    np.testing.assert_array_equal(v, t.values)


def test_scales_are_bf16_and_errors_within_half_a_step():
    w = S._rng(2, "w4").standard_normal((16, 512)).astype(np.float32)
    t = S.quantize_groups_w4(w)
    np.testing.assert_array_equal(S.bf16_bits_to_f32(S.to_bf16_bits(t.scale)), t.scale)
    step = np.repeat(t.scale.astype(np.float64), 64, axis=1)
    # the scale rounds by at most 2^-8 of itself: codes stay within 7 (1 + 2^-8), which rounds to 7
    assert np.all(np.abs(t.values - w) <= step / 2 + 1e-12 + 7 * step * 2.0 ** -8)
    assert unpack(t.q).max() <= 7 and unpack(t.q).min() >= -8


def test_ties_go_to_even_and_zero_groups_to_zero():
    w = np.zeros((2, 128), np.float32)
    w[0, :5] = [7.0, 0.5, 1.5, -0.5, -2.5]     # scale 1
    t = S.quantize_groups_w4(w)
    assert t.scale[0, 0] == 1.0 and list(unpack(t.q)[0, :5]) == [7, 0, 2, 0, -2]
    assert np.all(t.values[1] == 0) and np.all(t.scale[1] == 1.0)
