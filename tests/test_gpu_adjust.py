"""dflash2_adjust_logits against the definition in 64 bits.

Tolerance: the steps are a division or product, a product of frequency and count, two subtractions and an addition in
fp32, each rounding by 2^-24 of its result (the count's conversion is exact); results are at most the sum S of the
terms' magnitudes, so 6 * 2^-24 * S bounds them, and a bfloat16 result adds 2^-8 of itself."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import operator_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_speculative_decoding_dflash2_gb300 import binding
    binding.lib()
    return binding


def dev(x, dtype):
    return None if x is None else torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


class Case:
    def __init__(self, batch, rows, vocab, dtype, history, seed=0, n_bias=0, masked=False, path=True, hot=None):
        rng = np.random.default_rng(seed)
        hot = min(vocab, hot or vocab)
        self.shape = (batch, rows, vocab)
        self.z = torch.from_numpy(rng.standard_normal(self.shape).astype(np.float32) * 4).to(dtype)
        self.tokens = rng.integers(0, hot, (batch, max(history, 1)))
        self.n = rng.integers(0, history + 1, batch)
        self.prompt = np.array([rng.integers(0, n + 1) for n in self.n])
        self.path = rng.integers(0, hot, (batch, rows - 1)) if path and rows > 1 else None
        self.rho = rng.uniform(0.7, 1.6, batch).astype(np.float32)
        self.presence, self.frequency = (rng.uniform(-1, 2, batch).astype(np.float32) for _ in range(2))
        self.bias_id = rng.integers(0, hot, (batch, n_bias)) if n_bias else None
        self.bias = rng.standard_normal((batch, n_bias)).astype(np.float32) * 5 if n_bias else None
        self.bits = rng.random(self.shape) < 0.7 if masked else None

    def words(self):
        if self.bits is None:
            return None
        b, r, v = self.shape
        w = -(-v // 32)
        full = np.ones((b, r, w * 32), bool)
        full[..., :v] = self.bits
        return np.packbits(full.reshape(b, r, w, 32), axis=3, bitorder="little").view(np.int32)[..., 0]

    def reference(self):
        b, r, v = self.shape
        z = self.z.double().numpy()
        out, size = np.empty_like(z), np.empty_like(z)
        for s in range(b):
            bias = [] if self.bias_id is None else list(zip(self.bias_id[s].tolist(), self.bias[s].astype(np.float64)))
            for i in range(r):
                drafts = [] if self.path is None else self.path[s, :i].tolist()
                args = (self.tokens[s, :self.n[s]].tolist(), int(self.prompt[s]), drafts)
                rest = (bias, None if self.bits is None else self.bits[s, i])
                out[s, i] = R.adjust(z[s, i], *args, float(self.rho[s]), float(self.presence[s]),
                                     float(self.frequency[s]), *rest)
                # (magnitudes: the terms without their signs)
                size[s, i] = R.adjust(np.abs(z[s, i]) * 2, *args, 1.0, -abs(float(self.presence[s])),
                                      -abs(float(self.frequency[s])), [(t, abs(w)) for t, w in bias], None)
        return out, size

    def run(self, B, pad=0, offset=0, in_place=False, status=0, **over):
        b, r, v = self.shape
        wide = v + pad
        buf = torch.full((b * r * wide + offset + 64,), 5.0, dtype=self.z.dtype, device="cuda")
        logits = buf[offset:offset + b * r * wide].view(b, r, wide)[..., :v]
        logits.copy_(self.z)
        if in_place:
            out = logits
        else:
            obuf = torch.full_like(buf, 6.0)
            out = obuf[offset:offset + b * r * wide].view(b, r, wide)[..., :v]
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        args = dict(prompt_len=dev(self.prompt, torch.int32), path=dev(self.path, torch.int32),
                    repetition=dev(self.rho, torch.float32), presence=dev(self.presence, torch.float32),
                    frequency=dev(self.frequency, torch.float32), bias_id=dev(self.bias_id, torch.int32),
                    bias=dev(self.bias, torch.float32), mask=dev(self.words(), torch.int32), workspace=ws)
        args.update(over)
        B.dflash2_adjust_logits(logits, dev(self.tokens, torch.int32), dev(self.n, torch.int32), out, **args)
        torch.cuda.synchronize()
        assert B.dflash2_read_device_status(ws) == status
        whole = (buf if in_place else obuf)
        mark = 5.0 if in_place else 6.0
        assert (whole[:offset] == mark).all() and (whole[offset + b * r * wide:] == mark).all()
        if pad:
            assert (whole[offset:offset + b * r * wide].view(b, r, wide)[..., v:] == mark).all()
        return out.double().cpu().numpy()

    def check(self, B, **kw):
        got = self.run(B, **kw)
        want, size = self.reference()
        gone = np.isneginf(want)
        assert np.array_equal(np.isneginf(got), gone)
        tol = 6 * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(want) if self.z.dtype == torch.bfloat16 else 0)
        bad = ~gone & ~(np.abs(got - np.where(gone, 0, want)) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])
        return got


TYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,rows,vocab,history,n_bias,masked,hot", [
    (1, 1, 1, 3, 0, False, None), (1, 1, 31, 0, 0, True, None), (2, 8, 500, 40, 5, True, 60),
    (3, 8, 1000, 300, 40, False, 1000), (2, 5, 12345, 2000, 300, True, 400), (1, 32, 4097, 700, 3, True, 50),
    (5, 3, 50257, 100, 1, False, 200), (1, 9, 20000, 5000, 65535, True, None), (40, 2, 3008, 64, 8, True, None)])
def test_rows(B, dtype, batch, rows, vocab, history, n_bias, masked, hot):
    Case(batch, rows, vocab, dtype, history, seed=vocab, n_bias=n_bias, masked=masked, hot=hot).check(B)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 0), (16, 3), (1, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_strides_and_borders(B, dtype, pad, offset, in_place):
    Case(2, 9, 777, dtype, 50, seed=pad, n_bias=9, masked=True, hot=100).check(B, pad=pad, offset=offset, in_place=in_place)


@pytest.mark.parametrize("dtype", TYPES)
def test_settings_left_out(B, dtype):
    c = Case(3, 4, 600, dtype, 30, seed=1, n_bias=4, masked=True, hot=40)
    c.rho[:], c.presence[:], c.frequency[:], c.prompt[:] = 1, 0, 0, 0
    c.check(B, repetition=None, presence=None, frequency=None, prompt_len=None)
    c.bits = c.bias_id = c.bias = None
    assert np.array_equal(c.run(B, repetition=None), c.z.double().numpy())
    c.path = None  # rows that all follow the same tokens
    c.presence[:] = 0.5
    c.check(B)


def test_the_last_of_an_ids_biases_counts_and_unused_entries_do_not(B):
    c = Case(1, 2, 300, torch.float32, 0, seed=2, n_bias=6)
    c.bias_id = np.array([[7, -1, 9, 7, -1, 9]])
    got = c.run(B)
    z = c.z.double().numpy()
    assert c.path[0, 0] not in (7, 9)
    assert np.allclose(got[0, :, 7] - z[0, :, 7], c.bias[0, 3], atol=1e-5)
    assert np.allclose(got[0, :, 9] - z[0, :, 9], c.bias[0, 5], atol=1e-5)
    # besides those, row 1 counts the draft before it
    assert {tuple(x) for x in np.argwhere(got != z)} == {(0, r, v) for r in (0, 1) for v in (7, 9)} | {(0, 1, int(c.path[0, 0]))}


def test_drafts_count_row_by_row(B):
    c = Case(1, 4, 100, torch.float32, 0, seed=3)
    c.path = np.array([[5, -1, 5]])
    c.rho[:], c.presence[:], c.frequency[:] = 1, 1.0, 0.25
    d = c.z.double().numpy() - c.check(B)
    assert np.allclose(d[0, :, 5], [0, 1.25, 1.25, 1.5], atol=1e-5) and np.abs(np.delete(d, 5, 2)).max() == 0


def test_infinities_stay_where_they_are(B):
    c = Case(1, 3, 200, torch.float32, 50, seed=4, masked=True, hot=200)
    c.z[0, 0, :20], c.z[0, 1, 20:40] = float("-inf"), float("inf")
    got, want = c.run(B), c.reference()[0]
    assert np.array_equal(np.isinf(got), np.isinf(want)) and np.array_equal(got[np.isinf(got)], want[np.isinf(want)])


def test_a_mask_without_a_bit(B):
    c = Case(1, 2, 333, torch.bfloat16, 20, seed=5, masked=True, n_bias=3)
    c.bits[:] = False
    assert np.isneginf(c.run(B)).all()


def test_bad_tokens_and_lengths_are_recorded(B):
    c = Case(2, 3, 400, torch.float32, 10, seed=6, n_bias=4, hot=30)
    c.n[:] = 10
    c.prompt[:] = 0
    good = c.check(B)
    for name, at in (("tokens", (0, 3)), ("path", (1, 0)), ("bias_id", (0, 1))):
        keep = getattr(c, name).copy()
        for bad in (400, 2 ** 31 - 1, -2, -2 ** 31):
            getattr(c, name)[at] = bad
            got = c.run(B, status=B.DEV_BAD_TOKEN)
            assert np.array_equal(got[1 - at[0]], good[1 - at[0]])
        setattr(c, name, keep)
    c.n[:] = [11, 10]
    assert np.array_equal(c.run(B, status=B.DEV_BAD_LENGTH), good)
    c.n[:] = [-5, 10]
    assert np.array_equal(c.run(B, status=B.DEV_BAD_LENGTH)[1], good[1])


def test_same_bits_again_and_captured(B):
    """Counts come from atomics, whose order does not show; a graph follows its inputs."""
    c = Case(3, 8, 5000, torch.bfloat16, 3000, seed=7, n_bias=50, masked=True, hot=90)
    first = c.run(B)
    assert np.array_equal(c.run(B), first)
    z, tok, n = c.z.cuda(), dev(c.tokens, torch.int32), dev(c.n, torch.int32)
    out, path, presence = torch.empty_like(z), dev(c.path, torch.int32), dev(c.presence, torch.float32)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        B.dflash2_adjust_logits(z, tok, n, out, path=path, presence=presence)
    for seed in (8, 9):
        c = Case(3, 8, 5000, torch.bfloat16, 3000, seed=seed, hot=90)
        c.rho[:], c.frequency[:], c.prompt[:] = 1, 0, 0
        for t, x in ((z, c.z), (tok, c.tokens), (n, c.n), (path, c.path), (presence, c.presence)):
            t.copy_(torch.as_tensor(x))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), c.run(B, repetition=None, frequency=None))
