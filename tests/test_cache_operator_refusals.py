"""Argument checks of the paged-cache operators, the attention over a paged cache and the changes to logits: all of them
happen on the host before anything is launched, so they are tested without a GPU, on addresses that are never read."""

import ctypes

import pytest

P = 1 << 20  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def B():
    pytest.importorskip("torch")
    from block_speculative_decoding_dflash2_gb300 import binding
    try:
        binding.lib()
    except ImportError as e:
        pytest.skip(str(e))
    return binding


def cache_of(B, dtype=1, n_pages=4, page=16, nkv=2, d=128, k=P, v=P, ke=None, ve=None):
    return ctypes.byref(B.Cache(dtype, n_pages, page, nkv, d, k, v, ke, ve))


@pytest.mark.parametrize("read", [False, True])
def test_cache_rows(B, read):
    f = B.lib().dflash2_cache_read if read else B.lib().dflash2_cache_append

    def call(cache="default", table=P, pages=4, batch=2, at=P, n=3, k=P, ks=256, v=P, vs=256, off=P, ws=None, **over):
        c = cache_of(B, **over) if cache == "default" else cache
        return f(c, table, pages, batch, at, n, off, k, ks, v, vs, ws, None) if read else \
            f(c, table, pages, batch, at, n, k, ks, v, vs, off, ws, None)

    assert call(cache=None) == -1
    for dtype in (0, 2, 3, 5, -1):
        assert call(dtype=dtype) == -4
    for over in (dict(d=96), dict(d=0), dict(nkv=0), dict(nkv=257), dict(page=0), dict(page=-16), dict(n_pages=0)):
        assert call(**over) == -2, over
    assert call(k=None) == -1 and call(v=None) == -1 and call(k=P + 8) == -1 and call(v=P + 2) == -1
    assert call(cache=cache_of(B, k=None)) == -1 and call(cache=cache_of(B, v=P + 4)) == -1
    assert call(cache=cache_of(B, dtype=4)) == -1 and call(cache=cache_of(B, dtype=4, ke=P)) == -1
    assert call(table=None) == -1 and call(table=P + 2) == -1 and call(pages=0) == -2 and call(batch=0) == -2
    assert call(batch=65536) == -2 and call(pages=2 ** 27, page=16) == -2 and call(n=-1) == -2
    assert call(off=None) == -1 and call(off=P + 1) == -1 and call(at=P + 2) == -1
    if not read:
        assert call(at=None) == -1
    assert call(ks=255) == -2 and call(vs=248) == -2 and call(ks=260) == -2 and call(vs=-256) == -2
    assert call(ws=P + 2) == -5
    assert call(n=0) == 0 and call(n=0, k=None, v=None) == 0


def test_attend(B):
    f, size = B.lib().dflash2_attend, B.lib().dflash2_attend_workspace

    def call(cache="default", table=P, pages=4, batch=2, n_tok=3, n_new=None, kv=P, nq=4, q=P, qs=512, out=P, os_=512,
             scale=0.1, causal=1, window=0, shared=0, ws=P, wsb=1 << 40, **over):
        c = cache_of(B, **over) if cache == "default" else cache
        return f(c, table, pages, batch, n_tok, n_new, kv, nq, q, qs, out, os_, scale, causal, window, shared, ws, wsb, None)

    assert call(cache=None) == -1 and call(dtype=0) == -4 and call(d=32) == -2 and call(dtype=4) == -1
    assert call(table=None) == -1 and call(kv=None) == -1 and call(q=None) == -1 and call(out=None) == -1
    assert call(q=P + 8) == -1 and call(out=P + 4) == -1 and call(kv=P + 2) == -1 and call(n_new=P + 1) == -1
    assert call(n_tok=0) == -2 and call(n_tok=1025) == -2 and call(nq=3) == -2 and call(nq=0) == -2 and call(nq=1026) == -2
    assert call(window=-1) == -2 and call(shared=-1) == -2 and call(shared=65) == -2
    assert call(qs=511) == -2 and call(os_=504) == -2 and call(qs=516) == -2 and call(os_=-512) == -2
    for scale in (0.0, -0.1, float("nan"), float("inf")):
        assert call(scale=scale) == -1, scale
    need = size(cache_of(B), 2, 3, 4, 0)
    assert need >= 256 and call(ws=None) == -5 and call(ws=P + 8) == -5 and call(wsb=need - 1) == -5
    assert size(cache_of(B), 2, 3, 4, 64) > need
    for bad in ((0, 3, 4, 0), (65536, 3, 4, 0), (2, 0, 4, 0), (2, 1025, 4, 0), (2, 3, 3, 0), (2, 3, 4, -1)):
        assert size(cache_of(B), *bad) == 0, bad
    assert size(None, 2, 3, 4, 0) == 0 and size(cache_of(B, nkv=0), 2, 3, 4, 0) == 0


def test_adjust_logits(B):
    f = B.lib().dflash2_adjust_logits

    def call(dt=0, batch=2, rows=3, vocab=10, z=P, stride=10, tok=P, most=5, n=P, prompt=None, path=None, rho=None,
             pres=None, freq=None, bid=None, bias=None, nb=0, mask=None, out=P, os_=10, ws=None):
        return f(dt, batch, rows, vocab, z, stride, tok, most, n, prompt, path, rho, pres, freq, bid, bias, nb, mask, out,
                 os_, ws, None)

    assert call(dt=2) == -4 and call(dt=4) == -4 and call(batch=0) == -2 and call(rows=0) == -2 and call(vocab=0) == -2
    assert call(vocab=(1 << 20) + 1, stride=1 << 21, os_=1 << 21) == -2 and call(batch=65536, rows=1) == -2
    assert call(stride=9) == -2 and call(os_=9) == -2 and call(most=-1) == -2 and call(nb=-1) == -2 and call(nb=65536) == -2
    assert call(z=None) == -1 and call(out=None) == -1 and call(z=P + 2) == -1 and call(out=P + 2) == -1
    assert call(dt=1, z=P + 1) == -1 and call(tok=None) == -1 and call(n=None) == -1
    assert call(nb=3) == -1 and call(nb=3, bid=P) == -1 and call(nb=3, bias=P) == -1
    assert call(path=P, rows=1) == -3 and call(path=P, rows=33) == -3
    for name in ("tok", "n", "prompt", "path", "rho", "pres", "freq", "mask"):
        assert call(**{name: P + 2}) == -1, name
    assert call(z=P, out=P, stride=12, os_=10) == -2  # in place, but not row upon row
    assert call(ws=P + 1) == -5


def test_binding_refuses_what_it_cannot_pass(B):
    import torch
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn

    def status(fn, *a, **k):
        with pytest.raises(B.DFlash2Error) as e:
            fn(*a, **k)
        return e.value.status

    k = torch.zeros((2, 16, 2, 64), dtype=bf)
    assert status(B.PagedCache, k, k) == -1  # on the host
    assert status(B.PagedCache, k.float(), k.float()) == -4 and status(B.PagedCache, k, k.to(f8)) == -4
    assert status(B.PagedCache, k, k[:1]) == -2 and status(B.PagedCache, k[0], k[0]) == -2
    assert status(B.PagedCache, k.transpose(1, 2), k.transpose(1, 2)) == -2
    z = torch.zeros((1, 2, 10))
    assert status(B.dflash2_adjust_logits, z, None, None, z) == -1


@pytest.mark.gpu
def test_binding_refuses_types_shapes_and_layouts(B):
    import torch
    c = dict(device="cuda")
    bf, i32 = torch.bfloat16, torch.int32

    def status(fn, *a, **k):
        with pytest.raises(B.DFlash2Error) as e:
            fn(*a, **k)
        return e.value.status

    pool = torch.zeros((4, 16, 2, 64), dtype=bf, **c)
    assert status(B.PagedCache, pool, pool, torch.zeros((4, 16, 2), dtype=torch.uint8, **c)) == -1
    p8 = pool.to(torch.float8_e4m3fn)
    ex = torch.zeros((4, 16, 2), dtype=torch.uint8, **c)
    assert status(B.PagedCache, p8, p8) == -1 and status(B.PagedCache, p8, p8, ex, ex[:2]) == -2
    assert status(B.PagedCache, p8, p8, ex, ex.to(i32)) == -4
    cache = B.PagedCache(pool, pool.clone())
    table, one, off = torch.zeros((1, 4), dtype=i32, **c), torch.zeros((1,), dtype=i32, **c), torch.zeros((2,), dtype=i32, **c)
    x = torch.zeros((3, 2, 64), dtype=bf, **c)
    ap = B.dflash2_cache_append
    assert status(ap, cache, table, one, x.float(), x, off) == -4 and status(ap, cache, table, one, x[:, :1], x, off) == -2
    assert status(ap, cache, table, one, x, x[:2], off) == -2 and status(ap, cache, table, one, x, x, off[:1]) == -2
    assert status(ap, cache, table[0], one, x, x, off) == -2 and status(ap, cache, table.long(), one, x, x, off) == -4
    assert status(ap, cache, table, one, x.transpose(1, 2).contiguous().transpose(1, 2), x, off) == -2
    assert status(ap, cache, table, one, x, x, off, torch.zeros(8, dtype=torch.uint8, **c)) == -5
    assert status(ap, cache, table, None, x, x, off) == -1 and status(ap, cache, table, one, x, x, None) == -1
    odd = torch.zeros((3 * 132,), dtype=bf, **c)
    assert status(ap, cache, table, one, odd.as_strided((3, 2, 64), (132, 64, 1)), x, off) == -2
    assert status(ap, cache, table, one, odd[4:].as_strided((2, 2, 64), (128, 64, 1)), x[:2], off) == -1
    q = torch.zeros((1, 2, 4, 64), dtype=bf, **c)
    ws = torch.zeros(B.dflash2_attend_workspace(cache, 1, 2, 4), dtype=torch.uint8, **c)
    at = B.dflash2_attend
    assert status(at, cache, table, one, q, q.clone(), None) == -5 and status(at, cache, table, one, q, q.clone(), ws[:64]) == -5
    assert status(at, cache, table, one, q.half(), q.clone(), ws) == -4 and status(at, cache, table, one, q, q[:, :1], ws) == -2
    assert status(at, cache, table, one, q[0], q[0], ws) == -2 and status(at, cache, table, one, q[..., :32], q[..., :32], ws) == -2
    assert status(at, cache, table, one, q.expand(2, 2, 4, 64), q, ws) == -2
    assert status(at, cache, table, one, q, q.clone(), ws, scale=0.0) == -1
    assert status(at, cache, table, one, q, q.clone(), ws, shared_len=65) == -2
    z = torch.zeros((2, 3, 40), **c)
    tok, n = torch.zeros((2, 5), dtype=i32, **c), torch.zeros((2,), dtype=i32, **c)
    ad = B.dflash2_adjust_logits
    assert status(ad, z, tok, n, z.to(bf)) == -4 and status(ad, z, tok, n, z[:, :2]) == -2
    assert status(ad, z, tok[0], n, z.clone()) == -2 and status(ad, z, tok, n[:1], z.clone()) == -2
    assert status(ad, z, tok.long(), n, z.clone()) == -4 and status(ad, z, tok, n, z.clone(), path=tok) == -2
    assert status(ad, z, tok, n, z.clone(), mask=torch.zeros((2, 3, 1), dtype=i32, **c)) == -2
    assert status(ad, z, tok, n, z.clone(), bias_id=tok) == -1
    assert status(ad, z, tok, n, z.clone(), bias_id=tok, bias=z[0, :2, :5].contiguous().to(bf)) == -4
    assert status(ad, z, tok, n, z.clone(), repetition=n) == -4
