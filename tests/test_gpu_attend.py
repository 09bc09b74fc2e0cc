"""dflash2_attend against the 64-bit form, row by row.

Tolerance of a value, from the roundings: the result's own to bfloat16 (2^-8 of it, finfo.eps / 2), and the weights'
against each other.  A weight is formed from a score with errors of about 2^-23 of the sum of its products' magnitudes
(at most 2^6 in these inputs, so 2^-17) and held with 2^-9 (8-bit caches on the tensor cores: nine bits) or 2^-15
(otherwise): relative to the sum of weight times |value|, 2^-9 + 2^-16 and 2^-14."""

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


@pytest.fixture(autouse=True, params=[0, 2], ids=["choice", "tensor"])
def kernel(request, B):
    """The library's choice of a kernel, and the tensor cores' for short sequences too."""
    B.dflash2_test_force_attend(request.param)
    yield
    B.dflash2_test_force_attend(0)


class Case:
    """A pool with the sequences' pages in random order, everything else in it NaN (bfloat16) or NaN codes."""

    def __init__(self, B, cache, d, page, nq, nkv, n_tok, lens, shared=0, n_new=None, seed=0, spread=2.0):
        rng = np.random.default_rng(seed)
        self.B, self.cache_type, self.d, self.page, self.shared = B, cache, d, page, shared
        self.nq, self.nkv, self.n_tok, self.lens = nq, nkv, n_tok, list(lens)
        self.count = [n_tok] * len(lens) if n_new is None else list(n_new)
        batch, first = len(lens), -(-shared // page)
        own = [max(0, -(-n // page) - first) for n in lens]
        order = rng.permutation(first + sum(own) + 2)
        self.table = np.full((batch, max(1, first + max(own))), -1 if shared == 0 else 0, np.int32)
        at = first
        for i, n in enumerate(own):
            self.table[i, :first] = order[:first]
            self.table[i, first:first + n] = order[at:at + n]
            at += n
        shape = (order.size, page, nkv, d)
        self.pool = {}
        for name in ("k", "v"):
            x = torch.full(shape, float("nan"), dtype=torch.bfloat16)
            vals = torch.from_numpy(rng.standard_normal(shape, np.float32)) * (1.0 if name == "k" else spread)
            if name == "v":
                vals *= torch.from_numpy(np.exp2(rng.integers(-6, 3, shape[:3])).astype(np.float32))[..., None]
            vals = vals.to(torch.bfloat16)
            for i in range(batch):
                for p in range(lens[i]):
                    pg = self.table[i, p // page]
                    x[pg, p % page] = vals[pg, p % page]
            self.pool[name] = x
        self.q = torch.from_numpy(rng.standard_normal((batch, n_tok, nq, d), np.float32)).to(torch.bfloat16)
        self.quantise()

    def quantise(self):
        self.vals, self.dev = {}, {}
        for name, x in self.pool.items():
            if self.cache_type == "bf16":
                self.vals[name], self.dev[name] = x.double().numpy(), x.cuda()
                self.dev[name + "_exp"] = None
                continue
            # (the format's own rounding is tested elsewhere: here torch's conversion of scaled values serves)
            top = torch.where(torch.isfinite(x), x.abs().float(), 0.0).amax(-1)
            e = torch.clamp(torch.ceil(torch.log2(torch.clamp(top, min=1e-30) / 448)), -100, 100)
            codes = (x.float() / torch.exp2(e)[..., None]).to(torch.float8_e4m3fn)
            exps = (e + 127).to(torch.uint8)
            self.vals[name] = codes.double().numpy() * np.exp2(exps.numpy()[..., None] - 127.0)
            self.dev[name], self.dev[name + "_exp"] = codes.cuda(), exps.cuda()

    def reference(self, scale, causal, window):
        out, mag = np.zeros(tuple(self.q.shape)), np.zeros(tuple(self.q.shape))
        for i, n in enumerate(self.count):
            rows = [(self.table[i, p // self.page], p % self.page) for p in range(self.lens[i])]
            k, v = (np.array([self.vals[x][r] for r in rows]).reshape(-1, self.nkv, self.d) for x in ("k", "v"))
            out[i, :n], mag[i, :n] = R.attend(self.q[i, :n].double().numpy(), k, v, scale, causal, window)
        return out, mag

    def run(self, scale=None, causal=True, window=0, stride=0, stream=None, status=0):
        B = self.B
        cache = B.PagedCache(self.dev["k"], self.dev["v"], self.dev["k_exp"], self.dev["v_exp"])
        batch = len(self.lens)
        ws = torch.zeros(B.dflash2_attend_workspace(cache, batch, self.n_tok, self.nq, self.shared), dtype=torch.uint8,
                         device="cuda")
        ws[256:] = 0xff  # only the status word needs zeros
        wide = self.nq * self.d + stride
        q = torch.full((batch, self.n_tok, wide), float("nan"), dtype=torch.bfloat16, device="cuda")
        out = torch.full_like(q, 7.0)
        qv, ov = (x[..., :self.nq * self.d].unflatten(2, (self.nq, self.d)) for x in (q, out))
        qv.copy_(self.q)
        n_new = None
        if self.count != [self.n_tok] * batch:
            n_new = torch.tensor(getattr(self, "passed", self.count), dtype=torch.int32, device="cuda")
            for i, n in enumerate(self.count):
                qv[i, n:] = float("nan")
        B.dflash2_attend(cache, torch.from_numpy(self.table).cuda(), torch.tensor(self.lens, dtype=torch.int32,
                         device="cuda"), qv, ov, ws, n_new=n_new, scale=scale, causal=causal, window=window,
                         shared_len=self.shared, stream=stream)
        torch.cuda.synchronize()
        assert B.dflash2_read_device_status(ws) == status
        if stride:
            assert (out[..., self.nq * self.d:] == 7).all()
        for i, n in enumerate(self.count):
            assert (ov[i, n:] == 7).all(), "rows behind the sequence's tokens were written"
        return ov.double().cpu().numpy()

    def check(self, scale=None, causal=True, window=0, stride=0):
        got = self.run(scale, causal, window, stride)
        want, mag = self.reference(self.d ** -0.5 if scale is None else scale, causal, window)
        fast8 = self.cache_type == "e4m3" and self.d == 128 and self.page % 16 == 0
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -16 if fast8 else 2.0 ** -14) * mag + 1e-30
        for i, n in enumerate(self.count):
            bad = ~(np.abs(got[i, :n] - want[i, :n]) <= tol[i, :n])
            assert not bad.any(), (i, np.argwhere(bad)[:5].tolist(), got[i, :n][bad][:5], want[i, :n][bad][:5])
        return got


CACHES = ("bf16", "e4m3")


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d,page", [(128, 16), (128, 48), (64, 16), (128, 20)])
@pytest.mark.parametrize("nq,nkv,n_tok,lens", [
    (4, 1, 1, [1]), (4, 2, 1, [0, 1, 15, 16, 17, 127, 128, 129, 300]), (8, 2, 8, [8, 20, 130, 257]),
    (5, 5, 3, [700]), (40, 8, 16, [16, 150, 400]), (32, 1, 5, [40, 333]), (24, 2, 31, [31, 280])])
def test_causal(B, cache, d, page, nq, nkv, n_tok, lens):
    Case(B, cache, d, page, nq, nkv, n_tok, lens, seed=len(lens) + n_tok).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("nq,nkv,n_tok,lens,window", [
    (8, 2, 8, [9, 300], 0), (8, 2, 8, [9, 300, 515], 1), (8, 2, 8, [9, 300, 515], 130), (16, 1, 20, [20, 600], 33),
    (4, 4, 1, [1000, 3], 100)])
@pytest.mark.parametrize("causal", [True, False])
def test_windows_and_whole_blocks(B, cache, nq, nkv, n_tok, lens, window, causal):
    Case(B, cache, 128, 16, nq, nkv, n_tok, lens, seed=window).check(causal=causal, window=window)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("nq,nkv,n_tok,lens,shared", [
    (4, 2, 1, [200, 130], 128), (8, 2, 8, [300, 310, 500], 290), (8, 1, 16, [90, 400, 350], 64),
    (32, 2, 16, [600, 520, 700], 512), (4, 1, 2, [33, 60, 100, 500], 400), (4, 1, 1, [50] * 40, 49),
    (8, 1, 7, [1000] * 30, 992)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 150)])
def test_shared_prefix(B, cache, nq, nkv, n_tok, lens, shared, causal, window):
    if shared > min(lens):  # sequences that end inside the shared part: only their own positions count
        pass
    Case(B, cache, 128, 16, nq, nkv, n_tok, lens, shared=shared, seed=shared).check(causal=causal, window=window)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [128, 64])
def test_token_counts_out_of_range_are_recorded(B, cache, d):
    c = Case(B, cache, d, 16, 8, 2, 3, [50, 60, 70], n_new=[3, 0, 2], seed=12)
    want = c.check()
    c.passed = [7, -2, 2]  # counts as the nearer ends: 3 and 0
    assert np.array_equal(c.run(status=B.DEV_BAD_LENGTH), want)


@pytest.mark.parametrize("cache", CACHES)
def test_ragged_tokens(B, cache):
    for shared in (0, 64):
        Case(B, cache, 128, 16, 8, 2, 9, [200, 100, 90, 300], shared=shared, n_new=[9, 0, 1, 4]).check(stride=24)
    Case(B, cache, 64, 16, 8, 2, 9, [200, 100, 90, 300], n_new=[9, 0, 1, 4]).check(stride=24)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("lens,nq,nkv,n_tok", [([3000, 10, 2000], 4, 1, 2), ([8200], 2, 1, 1), ([70] * 300, 2, 1, 1),
                                               ([5000, 5000], 16, 1, 20), ([700], 2, 1, 200), ([40, 3] * 500, 2, 1, 1),
                                               ([66] * 210, 8, 1, 33), ([20, 700, 2] * 150, 8, 4, 2)])
def test_long_and_many(B, cache, lens, nq, nkv, n_tok):
    Case(B, cache, 128, 16, nq, nkv, n_tok, lens, seed=3).check()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("shared", [0, 160])
def test_wide_scores(B, cache, shared):
    """Scores of hundreds: references move, and most weights vanish."""
    c = Case(B, cache, 128, 16, 8, 2, 4, [900, 333], shared=shared, seed=9)
    # a score's error grows with it: 2^-23 of products of up to 8 * 16 * 11 in 2^-units, so weights are held to 2^-10
    got = c.run(scale=1.0)
    want, mag = c.reference(1.0, True, 0)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -10) * mag).all()


@pytest.mark.parametrize("cache", CACHES)
def test_heavy_key_over_a_long_flat_rest(B, cache):
    """One key with most of the mass, thousands with little each: together they must not be lost."""
    c = Case(B, cache, 128, 16, 4, 1, 1, [6000], seed=4)
    first = c.table[0, 0]
    c.q[:] = 0
    c.q[..., 0] = 8.0
    for i in range(6000):
        c.pool["k"][c.table[0, i // 16], i % 16, :, 0] = -8.0
        c.pool["v"][c.table[0, i // 16], i % 16] = 1.0
    c.pool["k"][first, 0, :, 0] = 8.0  # 2 * 64 / sqrt(128) above the others: e^11.3, 6000 of them are 0.07 of it
    c.pool["v"][first, 0] = -1.0
    c.quantise()
    got = c.check()
    assert (got > -0.88).all() and (got < -0.85).all()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [128, 64])
def test_what_a_token_does_not_see(B, cache, d):
    """NaN and infinities in keys that later tokens see do not reach earlier ones; tokens that see them are NaN."""
    c = Case(B, cache, d, 16, 8, 2, 6, [206, 128, 40], seed=5)
    clean = c.check()
    for i, n in enumerate(c.lens):
        for name in ("k", "v"):
            p = n - 2  # the key of the last token but one
            c.pool[name][c.table[i, p // 16], p % 16, :, 3] = float("nan" if name == "k" else "inf")
    c.quantise()
    got = c.run()
    assert np.array_equal(got[:, :4], clean[:, :4])
    assert np.isnan(got[:, 4:]).any(-1).all()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [128, 64])
def test_bad_pages_and_lengths(B, cache, d):
    """Keys on pages that do not exist are left out, and recorded; a length past the block table ends there."""
    c = Case(B, cache, d, 16, 4, 2, 2, [100, 300], seed=6)
    keep = c.table.copy()
    c.table[1, 5] = 10 ** 6
    c.table[1, 9] = -3
    got = c.run(status=B.DEV_BAD_PAGE)
    gone = set(range(80, 96)) | set(range(144, 160))
    rows = [(keep[1, p // 16], p % 16) for p in range(300)]
    for t in range(2):
        keys = [p for p in range(300 - 1 + t) if p not in gone]
        k, v = (np.array([c.vals[x][rows[p]] for p in keys]) for x in ("k", "v"))
        want, mag = R.attend(c.q[1, t:t + 1].double().numpy(), k, v, d ** -0.5, False, 0)
        assert (np.abs(got[1, t] - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -8.9 * mag[0]).all()
    c.table = keep
    c.lens = [100, 19 * 16]
    c.pool["k"][keep[1, 18], 12:] = 0
    c.pool["v"][keep[1, 18], 12:] = 0
    c.quantise()
    whole = c.run()
    c.lens = [100, 5000]
    assert np.array_equal(c.run(status=B.DEV_BAD_LENGTH), whole)


@pytest.mark.parametrize("cache", CACHES)
def test_same_bits_again_and_on_another_stream(B, cache):
    c = Case(B, cache, 128, 16, 8, 2, 8, [900, 77, 1500], shared=64, seed=8)
    one = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert np.array_equal(one, c.run())
    assert np.array_equal(one, c.run())


@pytest.mark.parametrize("cache", CACHES)
def test_captured_with_lengths_that_change(B, cache):
    """One graph, replayed with other lengths and tokens in the same buffers."""
    c = Case(B, cache, 128, 16, 8, 2, 4, [400, 300, 200], seed=11)
    cache_t = B.PagedCache(c.dev["k"], c.dev["v"], c.dev["k_exp"], c.dev["v_exp"])
    ws = torch.zeros(B.dflash2_attend_workspace(cache_t, 3, 4, 8, 0), dtype=torch.uint8, device="cuda")
    table, q = torch.from_numpy(c.table).cuda(), torch.zeros((3, 4, 8, 128), dtype=torch.bfloat16, device="cuda")
    out, lens = torch.zeros_like(q), torch.tensor([4, 4, 4], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        B.dflash2_attend(cache_t, table, lens, q, out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        B.dflash2_attend(cache_t, table, lens, q, out, ws)
    for seqs in ([400, 300, 200], [5, 0, 199], [130, 128, 4]):
        c.lens = seqs
        q.copy_(c.q)
        lens.copy_(torch.tensor(seqs, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), c.run()), seqs
    assert B.dflash2_read_device_status(ws) == 0


def test_random_calls(B):
    """Sizes drawn over the range, each against the reference."""
    rng = np.random.default_rng(77)
    for i in range(24):
        nkv, group = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 5, 8]))
        n_tok, batch = int(rng.integers(1, 20)), int(rng.integers(1, 6))
        lens = [int(x) for x in rng.integers(0, 700, batch)]
        shared = int(rng.integers(0, max(lens) + 1)) if rng.random() < 0.4 else 0
        n_new = [int(x) for x in rng.integers(0, n_tok + 1, batch)] if rng.random() < 0.4 else None
        c = Case(B, str(rng.choice(CACHES)), 128, int(rng.choice([16, 32])), nkv * group, nkv, n_tok, lens,
                 shared=shared, n_new=n_new, seed=1000 + i)
        c.check(causal=bool(rng.random() < 0.7), window=int(rng.integers(1, 300)) if rng.random() < 0.3 else 0)
