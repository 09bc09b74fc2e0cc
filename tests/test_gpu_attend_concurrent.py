"""dflash2_attend and the cache rows on two streams at once, each with a workspace of its own, eagerly and as two captured
graphs: the same bits as one after the other."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_speculative_decoding_dflash2_gb300 import binding
    binding.lib()
    return binding


class Work:
    """Rows appended behind 100 positions and attended over, by a batch of its own in a pool of its own."""

    def __init__(self, B, cache, batch, n_tok, keys, shared, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        nkv, nq, d, page = 2, 8, 128, 16
        self.B, self.n_tok, self.shared = B, n_tok, shared
        pages = -(-(keys + n_tok) // page)
        dtype = torch.bfloat16 if cache == "bf16" else torch.uint8
        pool = [torch.zeros((batch * pages, page, nkv, d), dtype=dtype, device="cuda") for _ in range(2)]
        exps = [None, None]
        if cache == "e4m3":
            pool = [x.view(torch.float8_e4m3fn) for x in pool]
            exps = [torch.ones((batch * pages, page, nkv), dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.cache = B.PagedCache(*pool, *exps)
        self.table = torch.randperm(batch * pages, generator=gen, device="cuda").to(torch.int32).view(batch, pages)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        draw = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
        B.dflash2_cache_append(self.cache, self.table, i32([0] * batch), draw(batch * keys, nkv, d),
                               draw(batch * keys, nkv, d), i32([keys * i for i in range(batch + 1)]))
        self.before, self.after = i32([keys] * batch), i32([keys + n_tok] * batch)
        self.off = i32([n_tok * i for i in range(batch + 1)])
        self.k, self.v, self.q = draw(batch * n_tok, nkv, d), draw(batch * n_tok, nkv, d), draw(batch, n_tok, nq, d)
        self.out = torch.zeros_like(self.q)
        self.back = [torch.zeros_like(self.k) for _ in range(2)]
        self.ws = torch.zeros(B.dflash2_attend_workspace(self.cache, batch, n_tok, nq, shared), dtype=torch.uint8,
                              device="cuda")

    def go(self):
        self.B.dflash2_cache_append(self.cache, self.table, self.before, self.k, self.v, self.off, self.ws)
        self.B.dflash2_attend(self.cache, self.table, self.after, self.q, self.out, self.ws, shared_len=self.shared)
        self.B.dflash2_cache_read(self.cache, self.table, self.before, self.off, *self.back, self.ws)

    def results(self):
        assert self.B.dflash2_read_device_status(self.ws) == 0
        return [t.clone() for t in (self.out, *self.back)]


@pytest.mark.parametrize("captured", [False, True])
def test_two_streams(B, captured):
    works = [Work(B, "bf16", 12, 6, 900, 0, 1), Work(B, "e4m3", 5, 16, 3000, 64, 2)]
    for w in works:
        w.go()
    torch.cuda.synchronize()
    alone = [w.results() for w in works]
    streams = [torch.cuda.Stream() for _ in works]
    graphs = []
    if captured:
        for w, s in zip(works, streams):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=s):
                w.go()
    for w in works:
        w.out.zero_()
        w.back[0].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (w, s) in enumerate(zip(works, streams)):
            with torch.cuda.stream(s):
                if captured:
                    graphs[i].replay()
                else:
                    w.go()
    torch.cuda.synchronize()
    for w, want in zip(works, alone):
        assert all(torch.equal(a, b) for a, b in zip(w.results(), want))
