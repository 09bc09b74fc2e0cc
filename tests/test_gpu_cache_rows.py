"""dflash2_cache_append and dflash2_cache_read against the format's definition: codes, exponent bytes and values are
compared exactly (the rows hold bfloat16 values, of which a code times a power of two is one again)."""

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


def make_cache(B, cache, n_pages, page, nkv, d):
    """A cache whose every byte is known: 0x55, which no test writes by chance."""
    shape = (n_pages, page, nkv, d)
    if cache == "bf16":
        k, v = (torch.full(shape, 7.25, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return B.PagedCache(k, v), (k, v, None, None)
    k, v = (torch.full(shape, 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ke, ve = (torch.full(shape[:3], 0x55, dtype=torch.uint8, device="cuda") for _ in range(2))
    return B.PagedCache(k, v, ke, ve), (k, v, ke, ve)


def rows_of(rng, n, nkv, d, kind="normal"):
    x = rng.standard_normal((n, nkv, d)).astype(np.float32) * np.exp2(rng.integers(-10, 10, (n, nkv, 1)))
    if kind == "edges":  # ties, largest and smallest magnitudes, zeros
        pool = np.array([0.0, -0.0, 448.0, 464.0, 480.0, 17.0, 19.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 1.0625, 1.1875,
                         3.3e38, -3.3e38, 1e-38, 1e-40, 2.0 ** -133, 1.75, 1.875, -448.0], np.float32)
        x = rng.choice(pool, (n, nkv, d))
        x[:, :, d // 2:] *= (rng.random((n, nkv, 1)) < 0.5)
        for i in range(n):  # rows of small values alone, too
            if i % 3 == 0:
                x[i] = np.where(np.abs(x[i]) > 2, 0, x[i])
            if i % 3 == 1:
                x[i] = np.where(np.abs(x[i]) > 1e-30, 0, x[i])
    return torch.from_numpy(x).to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def places(table, page, starts, counts):
    return [(table[s][(starts[s] + i) // page], (starts[s] + i) % page) for s in range(len(starts)) for i in range(counts[s])]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("nkv,d,page", [(1, 64, 16), (2, 128, 16), (3, 128, 20), (8, 128, 16), (8, 64, 1), (40, 128, 32)])
@pytest.mark.parametrize("starts,counts", [([0], [1]), ([5, 0, 31, 16], [3, 0, 40, 1]), ([100] * 37, [2] * 37)])
def test_rows_written_and_read_back(B, cache, nkv, d, page, starts, counts):
    rng = np.random.default_rng(nkv * d + page)
    need = [-(-(s + c) // page) for s, c in zip(starts, counts)]
    order = rng.permutation(sum(need) + 3).astype(np.int32)
    table = np.full((len(starts), max(need)), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    c, (pk, pv, ke, ve) = make_cache(B, cache, order.size, page, nkv, d)
    n = sum(counts)
    off = np.concatenate(([0], np.cumsum(counts)))
    rows = {"k": rows_of(rng, n, nkv, d), "v": rows_of(rng, n, nkv, d)}
    wide = {x: torch.zeros((n + 2, nkv * d + 8), dtype=torch.bfloat16, device="cuda") for x in rows}  # strided, rows behind
    for x in rows:
        wide[x][:n, :nkv * d] = rows[x].flatten(1).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    before = [None if t is None else t.view(torch.uint8).clone() for t in (pk, pv, ke, ve)]
    B.dflash2_cache_append(c, torch.from_numpy(table).cuda(), i32(starts), wide["k"][:, :nkv * d].unflatten(1, (nkv, d)),
                           wide["v"][:, :nkv * d].unflatten(1, (nkv, d)), i32(off), ws)
    torch.cuda.synchronize()
    assert B.dflash2_read_device_status(ws) == 0
    where = places(table, page, starts, counts)
    want = [None if t is None else t.cpu() for t in before]
    for j, (pg, o) in enumerate(where):
        for h in range(nkv):
            for x, (pool, exps) in (("k", (0, 2)), ("v", (1, 3))):
                if cache == "bf16":
                    want[pool][pg, o, h] = rows[x][j, h].contiguous().view(torch.uint8)
                else:
                    codes, b = R.quantise_row(rows[x][j, h].double().numpy()) if j < 6 else (None, None)
                    if codes is None:  # (rows beyond the first few: torch's conversion, as quick as that is slow)
                        _, b = top_byte(rows[x][j, h])
                        codes = (rows[x][j, h].float() * 2.0 ** (127 - b)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                    want[pool][pg, o, h] = torch.from_numpy(codes)
                    want[exps][pg, o, h] = b
    for got, w in zip((pk, pv, ke, ve), want):
        assert got is None or torch.equal(got.view(torch.uint8).cpu(), w)
    # back again, into strided rows with some behind that stay
    out = {x: torch.full((n + 2, nkv * d + 16), 3.0, dtype=torch.bfloat16, device="cuda") for x in rows}
    B.dflash2_cache_read(c, torch.from_numpy(table).cuda(), i32(starts), i32(off),
                         out["k"][:, :nkv * d].unflatten(1, (nkv, d)), out["v"][:, :nkv * d].unflatten(1, (nkv, d)), ws)
    torch.cuda.synchronize()
    assert B.dflash2_read_device_status(ws) == 0
    for x, (pool, exps) in (("k", (0, 2)), ("v", (1, 3))):
        got = out[x].cpu()
        assert (got[n:] == 3).all() and (got[:, nkv * d:] == 3).all()
        for j, (pg, o) in enumerate(where):
            if cache == "bf16":
                assert torch.equal(got[j, :nkv * d], rows[x][j].flatten())
            else:
                v = R.e4m3_values()[want[pool][pg, o].numpy()] * np.exp2(want[exps][pg, o].numpy()[:, None] - 127.0)
                assert np.array_equal(got[j, :nkv * d].double().numpy(), v.reshape(-1))


def top_byte(x):
    top = float(x.abs().max())
    return top, next(b for b in range(1, 256) if top <= 448 * 2.0 ** (b - 127))


def test_ties_ends_of_the_range_and_what_is_not_finite(B):
    rng = np.random.default_rng(0)
    x = rows_of(rng, 30, 2, 64, "edges")
    x[3, 0, 5], x[4, 1, 6], x[5, 0, 7], x[6, 0, :] = float("nan"), float("inf"), float("-inf"), float("nan")
    x[7, 1, :] = float("inf")
    c, (pk, _, ke, _) = make_cache(B, "e4m3", 3, 16, 2, 64)
    table = i32([[2, 0]])
    B.dflash2_cache_append(c, table, i32([0]), x.cuda(), x.cuda(), i32([0, 30]))
    torch.cuda.synchronize()
    codes, exps = pk.view(torch.uint8).cpu().numpy(), ke.cpu().numpy()
    for j in range(30):
        for h in range(2):
            want, b = R.quantise_row(x[j, h].double().numpy())
            got = codes[2 if j < 16 else 0, j % 16, h]
            assert exps[2 if j < 16 else 0, j % 16, h] == b, (j, h)
            nan = (want & 127) == 127
            assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], want[~nan]), (j, h)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_bad_pages_and_lengths(B, cache):
    c, (pk, pv, ke, ve) = make_cache(B, cache, 4, 16, 2, 64)
    before = pk.view(torch.uint8).clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    table = i32([[1, 7], [2, -1]])
    # sequence 0: positions 15 (page 1) and 16 (page 7: does not exist); sequence 1: 31 (page -1) and 32 (past the table)
    B.dflash2_cache_append(c, table, i32([15, 31]), x, x, i32([0, 2, 4]), ws)
    torch.cuda.synchronize()
    assert B.dflash2_read_device_status(ws) == B.DEV_BAD_PAGE | B.DEV_BAD_LENGTH
    changed = (pk.view(torch.uint8) != before).flatten(2).any(2).nonzero().tolist()
    assert changed == [[1, 15]]
    out = torch.full((5, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    B.dflash2_cache_read(c, table, i32([15, 31]), i32([0, 2, 4]), out, out.clone(), ws)
    torch.cuda.synchronize()
    assert B.dflash2_read_device_status(ws) == B.DEV_BAD_PAGE | B.DEV_BAD_LENGTH
    assert (out[0] == 1).all() and (out[1:4] == 0).all() and (out[4] == 9).all()


@pytest.mark.parametrize("batch", [1, 33, 1000, 5000])
def test_many_sequences(B, batch):
    """Rows of up to thousands of sequences, some without any, find their own."""
    rng = np.random.default_rng(batch)
    counts = rng.integers(0, 3, batch)
    counts[-1] = 1
    off = np.concatenate(([0], np.cumsum(counts)))
    n = int(off[-1])
    c, (pk, pv, _, _) = make_cache(B, "bf16", batch, 16, 1, 64)
    table = torch.from_numpy(rng.permutation(batch).astype(np.int32)[:, None].copy()).cuda()
    x = torch.arange(n, device="cuda").to(torch.bfloat16)[:, None, None].expand(n, 1, 64).contiguous()
    start = i32(rng.integers(0, 13, batch).tolist())
    B.dflash2_cache_append(c, table, start, x, -x, i32(off.tolist()))
    k, v = torch.empty_like(x), torch.empty_like(x)
    B.dflash2_cache_read(c, table, start, i32(off.tolist()), k, v)
    torch.cuda.synchronize()
    assert torch.equal(k, x) and torch.equal(v, -x)
    seq = torch.repeat_interleave(torch.arange(batch), torch.from_numpy(counts)).cuda()
    pos = start.long()[seq] + torch.arange(n, device="cuda") - torch.from_numpy(off).cuda()[seq]
    assert torch.equal(pk[table.long()[seq, 0], pos], x)


def test_captured(B):
    """One graph over rows and lengths that change between replays."""
    c, (pk, pv, ke, ve) = make_cache(B, "e4m3", 8, 16, 2, 128)
    table, start, off = i32([[0, 1], [2, 3]]), i32([0, 0]), i32([0, 2, 4])
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16, device="cuda")
    k, v = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        B.dflash2_cache_append(c, table, start, x, x, off)
        B.dflash2_cache_read(c, table, start, off, k, v)
    for at in (3, 17):
        x.copy_(torch.randint(-7, 8, x.shape, device="cuda").to(torch.bfloat16) * 8)  # four bits: exact
        start.fill_(at)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(k, x) and torch.equal(v, x)
