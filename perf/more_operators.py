"""Workloads of the operators around a target's verification pass: the paged cache in 8 bits (rows written, rows read
back), the attention that reads a paged cache, and the changes that a request's settings make to its logits.

Each operator has a plain form in elementary torch operations (``own`` false) and the library's call (``own`` true) on
the same inputs; ``exact`` gives the 64-bit result from the definition.

Definitions
  Paged cache: position p of sequence s lies in row p % page_size of page block_table[s][p // page_size]; a page holds
    page_size rows of n_kv_heads heads of head_dim values, keys and values each.
  8-bit cache: a head's row of values x is stored as e4m3 codes and one exponent byte b; a code c stands for
    c * 2^(b - 127).  b is the smallest byte >= 1 with max|x| <= 448 * 2^(b - 127) over the finite x; a code is the
    nearest e4m3 value of x * 2^(127 - b) (ties to even), NaN where x is not finite.
  Attention: the tokens of a call are the last ones of their sequence: token i of n sees the keys below
    kv_len - n + 1 + i, without causality all kv_len; with a window w only the last w of the keys that it sees.  The
    output is softmax(scale * q k) v over those keys, zeros where there is none.  Query head h reads key/value head
    h // (n_q_heads / n_kv_heads).  The first shared_len positions of all sequences lie in the same pages.
  Logits: a token counts as seen in row i of a sequence if it is among the sequence's tokens or the first i drafts; its
    count c is the number of times that it is among the tokens after the prompt and the first i drafts.  A seen
    token's logit z becomes z / repetition where z > 0, else z * repetition; then z - frequency * c, less presence
    where c > 0; then the token's bias is added (the last entry of an id counts); then tokens that the row's bit mask
    leaves out get -inf.
"""

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------------------------------------- cases

def _cache(op, name, cache, batch, lo, hi, nkv, d, page):
    c = {"op": op, "cache": cache, "batch": batch, "lo": lo, "hi": hi, "nkv": nkv, "d": d, "page": page}
    return dict(c, name=name) if name else c


def _attend(name, cache, batch, n_tok, lo, hi, nq, nkv, shared=0, d=128, page=16, causal=True, window=0, ragged=False):
    """lo .. hi: keys of a sequence after the shared ones, its own n_tok among them."""
    c = dict(_cache("attend", None, cache, batch, lo, hi, nkv, d, page), n_tok=n_tok, nq=nq, shared=shared,
             causal=causal, window=window, ragged=ragged)
    return dict(c, name=name) if name else c


def _adjust(name, batch, rows, vocab, dtype, history, n_bias, masked):
    c = {"op": "adjust", "batch": batch, "rows": rows, "vocab": vocab, "dtype": dtype, "history": history,
         "n_bias": n_bias, "masked": masked}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the rows of one verified block of the 8B-shaped target: latency alone
        _cache("append", "append_8", "e4m3", 1, 8, 8, 8, 128, 16),
        # 32 prompts of different lengths, written behind their first 100 positions
        _cache("append", "append_prompts", "e4m3", 32, 100, 2048, 8, 128, 16),
        # a short sequence read back, as when it moves to another batch
        _cache("read", "read_300", "e4m3", 1, 300, 300, 8, 128, 16),
        # the contexts of the 8B-shaped batch of 32 read back
        _cache("read", "read_contexts", "e4m3", 32, 512, 4096, 8, 128, 16),
        # plain decoding of one short sequence at the 8B shape: latency
        _attend("attend_1", "bf16", 1, 1, 300, 300, 32, 8),
        # a verification batch of the 8B shape: 32 requests, an anchor and seven drafts each
        _attend("attend_32x8", "bf16", 32, 8, 512, 4096, 32, 8),
        # the 27B shape's blocks of 16 on an 8-bit cache
        _attend("attend_8x16_e4m3", "e4m3", 8, 16, 8192, 8192, 40, 8),
        # the 30B-A3B shape's largest batch on an 8-bit cache, some requests with fewer drafts
        _attend("attend_256x7_e4m3", "e4m3", 256, 7, 8000, 8192, 32, 4, ragged=True),
        # 32 requests behind one long system prompt
        _attend("attend_shared_32x8", "bf16", 32, 8, 100, 600, 32, 8, shared=8192),
        # 64 requests of the 27B shape behind a long shared document, an 8-bit cache
        _attend("attend_shared_64x16_e4m3", "e4m3", 64, 16, 50, 500, 40, 8, shared=16384),
        # the verify rows of one request with a few thousand tokens behind it
        _adjust("adjust_8", 1, 8, 151936, "f32", 4000, 16, True),
        # the verify rows of 32 requests, bf16 logits as a readout stores them
        _adjust("adjust_256", 32, 8, 151936, "bf16", 4000, 64, True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.random()
    cache, page = rng.choice(("bf16", "e4m3")), rng.choice((16, 16, 16, 32, 64, 20))
    d = rng.choice((128, 128, 128, 64))
    if kind < 0.3:
        nkv = rng.choice((1, 2, 3, 4, 8))
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, min(8192, 700_000 // (batch * nkv)))
        return _cache(rng.choice(("append", "read")), None, cache, batch, _log(rng, 1, hi), hi, nkv, d, page)
    if kind < 0.75:
        nkv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 3, 4, 5, 8))
        n_tok, batch = rng.choice((1, 1, _log(rng, 2, 32), _log(rng, 2, 32))), _log(rng, 1, 128)
        rows = batch * n_tok * group * nkv
        shared = page * _log(rng, 1, max(1, min(16384, 600_000_000 // rows) // page)) if rng.random() < 0.35 else 0
        hi = _log(rng, n_tok, max(n_tok, min(8192, 3_000_000 // (batch * nkv))))
        return _attend(None, cache, batch, n_tok, _log(rng, n_tok, hi), hi, nkv * group, nkv, shared, d, page,
                       rng.random() < 0.8, _log(rng, 1, 4096) if rng.random() < 0.2 else 0, rng.random() < 0.3)
    vocab = _log(rng, 500, 151936)
    rows = rng.choice((1, rng.randint(2, 16)))
    batch = _log(rng, 1, max(1, min(256, 256 * 151936 // vocab) // rows))
    return _adjust(None, batch, rows, vocab, rng.choice(("f32", "bf16")), _log(rng, 1, 20000), rng.choice((0, 1, 300)),
                   rng.random() < 0.5)


def _lengths(case):
    """Row counts or key counts of the sequences, between lo and hi."""
    lo, hi = case["lo"], case["hi"]
    return [lo + int((hi - lo + 1) * ((0.5 + 0.6180339887 * i) % 1.0)) for i in range(case["batch"])]


def _tokens(case):
    """Tokens of each sequence in an attention call."""
    n = case["n_tok"]
    return [1 + (i * 5 + 2) % n if case["ragged"] else n for i in range(case["batch"])]


def _visible(case):
    """Keys that each (sequence, token) sees."""
    for own_keys, n in zip(_lengths(case), _tokens(case)):
        for i in range(n):
            keys = case["shared"] + own_keys - (n - 1 - i if case["causal"] else 0)
            yield min(keys, case["window"]) if case["window"] else keys


def work(case):
    if case["op"] == "adjust":
        n, v = case["batch"] * case["rows"], case["vocab"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2.0 * n * v * size + (n * v / 8 if case["masked"] else 0) + 4.0 * case["batch"] * case["history"],
                "flops": 1.0 * n * v}
    nkv, d = case["nkv"], case["d"]
    row = 2 * nkv * (2 * d if case["cache"] == "bf16" else d + 1)  # bytes of a position, keys and values
    if case["op"] != "attend":
        n = sum(_lengths(case))
        return {"bytes": n * (row + 4.0 * nkv * d), "flops": 4.0 * n * nkv * d}
    rows, keys = sum(_tokens(case)), case["shared"]
    for own_keys, n in zip(_lengths(case), _tokens(case)):
        keys += own_keys if not case["window"] else min(own_keys, case["window"] + n - 1)
    return {"bytes": keys * row + 4.0 * rows * case["nq"] * d, "flops": 4.0 * sum(_visible(case)) * case["nq"] * d}


# --------------------------------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _quantise(x):
    """[..., d] values -> e4m3 codes, exponent bytes (the definition above)."""
    x = x.float()
    m, e = torch.frexp(torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1))
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, -126, e).clamp_(-126, 127)
    half = torch.div(-e, 2, rounding_mode="floor")  # 2^-e may lie outside the range of a float: two factors
    y = torch.ldexp(torch.ldexp(x, half[..., None]), (-e - half)[..., None])
    y = torch.where(torch.isfinite(x), y, float("nan"))
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _pool(case, lengths, shared, g):
    """An empty cache pool with room for the sequences, and their block table: pages in random order, the shared ones
    first in every row."""
    page, nkv, d, batch = case["page"], case["nkv"], case["d"], case["batch"]
    first = shared // page
    each = [-(-(n + shared) // page) - first for n in lengths]
    order = torch.randperm(first + sum(each) + 3, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((batch, first + max(each)), dtype=torch.int32, device="cuda")
    table[:, :first] = order[:first]
    at = first
    for i, n in enumerate(each):
        table[i, first:first + n] = order[at:at + n]
        at += n
    shape = (order.numel(), page, nkv, d)
    if case["cache"] == "bf16":
        return {"k": torch.zeros(shape, dtype=torch.bfloat16, device="cuda"),
                "v": torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), "k_exp": None, "v_exp": None}, table
    codes, exps = (dict(dtype=torch.float8_e4m3fn, device="cuda"), dict(dtype=torch.uint8, device="cuda"))
    return {"k": torch.zeros(shape, **codes), "v": torch.zeros(shape, **codes),
            "k_exp": torch.full(shape[:3], 1, **exps), "v_exp": torch.full(shape[:3], 1, **exps)}, table


def _fill(pool, g):
    """Rows as a model leaves them: unit-variance keys, values of a scale that differs from row to row."""
    shape = pool["k"].shape
    for name in ("k", "v"):
        x = torch.randn(shape, generator=g, device="cuda")
        if name == "v":
            x *= torch.rand(shape[:3], generator=g, device="cuda")[..., None] + 0.5
        if pool["k_exp"] is None:
            pool[name].copy_(x)
        else:
            codes, exps = _quantise(x.to(torch.bfloat16))
            pool[name].view(torch.uint8).copy_(codes.view(torch.uint8))
            pool[name + "_exp"].copy_(exps)


def _cache_handle(s):
    from block_speculative_decoding_dflash2_gb300 import binding
    return binding.PagedCache(s["k"], s["v"], s["k_exp"], s["v_exp"])


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_rows(case, g):
    n, before = _lengths(case), 100 if case["batch"] > 1 else 0
    pool, table = _pool(case, [x + before for x in n], 0, g)
    off = [sum(n[:i]) for i in range(len(n) + 1)]
    shape = (off[-1], case["nkv"], case["d"])
    s = dict(pool, table=table, start=_i32([before] * len(n)), off=_i32(off), page=case["page"])
    if case["op"] == "read":
        _fill(pool, g)
        s["k_out"], s["v_out"] = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    else:
        scale = torch.rand(shape[:2], generator=g, device="cuda")[..., None] * 2 + 0.1
        s["k_new"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        s["v_new"] = (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)
    return s


def _prepare_attend(case, g):
    lengths, n_tok = _lengths(case), _tokens(case)
    pool, table = _pool(case, lengths, case["shared"], g)
    _fill(pool, g)
    shape = (case["batch"], case["n_tok"], case["nq"], case["d"])
    # scores of a standard deviation of 1.5: some keys count for much more than the others
    q = (torch.randn(shape, generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    ws = 64 << 20
    if own:
        from block_speculative_decoding_dflash2_gb300 import binding
        ws = binding.dflash2_attend_workspace(_cache_handle(pool), case["batch"], case["n_tok"], case["nq"],
                                              case["shared"])
    return dict(pool, table=table, kv_len=_i32([case["shared"] + n for n in lengths]), q=q, out=torch.zeros_like(q),
                n_new=_i32(n_tok) if case["ragged"] else None, scale=case["d"] ** -0.5, causal=case["causal"],
                window=case["window"], shared=case["shared"], page=case["page"],
                workspace=torch.zeros((ws,), dtype=torch.uint8, device="cuda"))


def _prepare_adjust(case, g):
    b, r, v = case["batch"], case["rows"], case["vocab"]
    z = torch.randn((b, r, v), generator=g, device="cuda") * 2.5
    uniform = lambda lo, hi: torch.rand((b,), generator=g, device="cuda") * (hi - lo) + lo  # noqa: E731
    most = case["history"]
    # text repeats itself: ids with a density that falls with the id
    ids = lambda *shape: (torch.rand(shape, generator=g, device="cuda").pow(3) * v).to(torch.int32).clamp_(max=v - 1)  # noqa: E731
    n = _i32([most - (i * 7) % (most // 3 + 1) for i in range(b)])
    s = {"logits": z if case["dtype"] == "f32" else z.to(torch.bfloat16), "tokens": ids(b, most), "n_tokens": n,
         "prompt_len": n // 3, "path": ids(b, r - 1) if r > 1 else None, "repetition": uniform(1.0, 1.3),
         "presence": uniform(0.0, 0.8), "frequency": uniform(0.0, 0.4), "bias_id": None, "bias": None, "mask": None}
    if case["n_bias"]:
        s["bias_id"] = ids(b, case["n_bias"])
        s["bias_id"][:, -1] = -1  # an entry that is not used
        s["bias"] = torch.randn((b, case["n_bias"]), generator=g, device="cuda") * 3
    if case["masked"]:
        s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (b, r, -(-v // 32)), generator=g, dtype=torch.int32, device="cuda")
    s["out"] = torch.empty_like(s["logits"])
    return s


def prepare(case, seed):
    g = _generator(seed)
    make = {"append": _prepare_rows, "read": _prepare_rows, "attend": _prepare_attend, "adjust": _prepare_adjust}
    s = dict(make[case["op"]](case, g), op=case["op"])
    if own and case["op"] != "adjust":
        s["cache"] = _cache_handle(s)
    return s


# ----------------------------------------------------------------------------------------------------- plain forms

def _row_places(s):
    """Rows of the pool (pages laid end to end) of the rows off[0] .. off[batch]."""
    off = s["off"].long()
    i = torch.arange((s["k_new"] if s["op"] == "append" else s["k_out"]).shape[0], device=off.device)
    seq = torch.searchsorted(off, i, right=True) - 1
    pos = s["start"].long()[seq] + i - off[seq]
    return s["table"].long()[seq, pos // s["page"]] * s["page"] + pos % s["page"]


def _plain_append(s):
    at = _row_places(s)
    for name in ("k", "v"):
        pool, x = s[name].flatten(0, 1), s[name + "_new"]
        if s["k_exp"] is None:
            pool[at] = x
        else:
            codes, exps = _quantise(x)
            pool.view(torch.uint8)[at] = codes.view(torch.uint8)
            s[name + "_exp"].flatten(0, 1)[at] = exps
    return {n: s[n] for n in ("k", "v", "k_exp", "v_exp") if s[n] is not None}


def _values(codes, exps, at):
    """fp32 values of the pool's rows (or pages) `at`."""
    if exps is None:
        return codes[at].float()
    return torch.ldexp(codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float(), exps[at].int()[..., None] - 127)


def _plain_read(s):
    at = _row_places(s)
    flat = {n: None if s[n] is None else s[n].flatten(0, 1) for n in ("k", "v", "k_exp", "v_exp")}
    return {n: _values(flat[n], flat[n + "_exp"], at).to(torch.bfloat16) for n in ("k", "v")}


def _plain_attend(s):
    b, n, nq, d = s["q"].shape
    nkv, table = s["k"].shape[2], s["table"].long()
    k, v = (_values(s[x], s[x + "_exp"], table).flatten(1, 2) for x in ("k", "v"))  # [b, keys, nkv, d]
    k, v = k.transpose(1, 2), v.transpose(1, 2)
    q = s["q"].float().view(b, n, nkv, nq // nkv, d).permute(0, 2, 3, 1, 4).reshape(b, nkv, nq // nkv * n, d)
    tok = torch.arange(n, device=q.device)
    count = torch.full((b,), n, device=q.device) if s["n_new"] is None else s["n_new"].long()
    top = s["kv_len"].long()[:, None] - (count[:, None] - 1 - tok) * int(s["causal"])  # [b, n]
    key = torch.arange(k.shape[2], device=q.device)
    seen = key < top[..., None]
    if s["window"]:
        seen &= key >= top[..., None] - s["window"]
    seen &= (tok < count[:, None])[..., None]
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(b, nkv, nq // nkv, n, -1)
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    x -= x.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = x.exp_()
    p /= p.sum(-1, keepdim=True).clamp_(min=1e-30)
    o = (p.view(b, nkv, nq // nkv * n, -1) @ v).view(b, nkv, nq // nkv, n, d).permute(0, 3, 1, 2, 4)
    return o.reshape(b, n, nq, d).to(torch.bfloat16)


def _plain_adjust(s):
    z = s["logits"].float()
    b, r, v = z.shape
    place = torch.arange(s["tokens"].shape[1], device=z.device)
    tokens = s["tokens"].long()
    there = place < s["n_tokens"][:, None]
    after = there & (place >= s["prompt_len"][:, None])
    zeros = lambda: torch.zeros((b, v), device=z.device)  # noqa: E731
    seen = zeros().scatter_add_(1, tokens, there.float())[:, None]
    count = zeros().scatter_add_(1, tokens, after.float())[:, None]
    if s["path"] is not None:
        drafts = torch.zeros_like(z).scatter_(2, torch.cat((s["path"][:, :1], s["path"]), 1).long()[..., None], 1.0)
        drafts[:, 0] = 0
        drafts = drafts.cumsum(1)
        seen, count = seen + drafts, count + drafts
    col = lambda p: s[p][:, None, None]  # noqa: E731
    z = torch.where(seen > 0, torch.where(z > 0, z / col("repetition"), z * col("repetition")), z)
    z = z - col("frequency") * count - col("presence") * (count > 0)
    if s["bias_id"] is not None:
        ids = s["bias_id"].long()
        rank = torch.arange(1, ids.shape[1] + 1, device=z.device).expand_as(ids)
        last = torch.zeros((b, v + 1), dtype=torch.int64, device=z.device)
        last.scatter_reduce_(1, torch.where(ids < 0, v, ids), rank, "amax")
        bias = torch.cat((torch.zeros_like(s["bias"][:, :1]), s["bias"]), 1).gather(1, last[:, :v])
        z = z + bias[:, None]
    if s["mask"] is not None:
        bit = torch.arange(32, device=z.device)
        keep = ((s["mask"][..., None] >> bit) & 1).flatten(2)[..., :v]
        z = torch.where(keep > 0, z, float("-inf"))
    return z.to(s["logits"].dtype)


# ------------------------------------------------------------------------------------------------- the library's

def _own(s):
    from block_speculative_decoding_dflash2_gb300 import binding as lib
    if s["op"] == "append":
        lib.dflash2_cache_append(s["cache"], s["table"], s["start"], s["k_new"], s["v_new"], s["off"])
        return {n: s[n] for n in ("k", "v", "k_exp", "v_exp") if s[n] is not None}
    if s["op"] == "read":
        lib.dflash2_cache_read(s["cache"], s["table"], s["start"], s["off"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if s["op"] == "attend":
        lib.dflash2_attend(s["cache"], s["table"], s["kv_len"], s["q"], s["out"], s["workspace"], n_new=s["n_new"],
                           scale=s["scale"], causal=s["causal"], window=s["window"], shared_len=s["shared"])
        return s["out"]
    lib.dflash2_adjust_logits(s["logits"], s["tokens"], s["n_tokens"], s["out"], prompt_len=s["prompt_len"],
                              path=s["path"], repetition=s["repetition"], presence=s["presence"],
                              frequency=s["frequency"], bias_id=s["bias_id"], bias=s["bias"], mask=s["mask"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    if state["op"] == "append":
        return _plain_append(state)
    if state["op"] == "read":
        return _plain_read(state)
    if state["op"] == "attend":
        return _plain_attend(state)
    return _plain_adjust(state)


# ------------------------------------------------------------------------------------------------- 64-bit results

def _exact_codes(x):
    """numpy float64 rows -> the e4m3 values of their codes, exponent bytes, from the definition."""
    top = np.abs(x).max(-1)
    b = np.full(top.shape, 1)
    for byte in range(255):  # the smallest byte that holds the row
        b = np.where(top > 448.0 * 2.0 ** (b - 127), byte + 1, b) if byte else b
    y = x / 2.0 ** (b - 127.0)[..., None]
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -20))), -6) - 3)
    return np.rint(y / step) * step, b


def _exact_rows(case, s):
    table, start, off = (s[n].cpu().numpy() for n in ("table", "start", "off"))
    page = case["page"]
    at = np.concatenate([table[i][p // page] * page + p % page for i in range(case["batch"])
                         for p in [start[i] + np.arange(off[i + 1] - off[i])]]).astype(np.int64)
    if case["op"] == "read":
        got = {}
        for n in ("k", "v"):
            x = s[n].flatten(0, 1).double().cpu().numpy()[at]
            got[n] = x if s["k_exp"] is None else x * 2.0 ** (s[n + "_exp"].flatten(0, 1).cpu().numpy()[at] - 127.0)[..., None]
        return got
    got = {}
    for n in ("k", "v"):
        pool, x = s[n].flatten(0, 1).double().cpu().numpy(), s[n + "_new"].double().cpu().numpy()
        if s["k_exp"] is not None:
            x, exps = _exact_codes(x)
            whole = s[n + "_exp"].flatten(0, 1).cpu().numpy().copy()
            whole[at] = exps
            got[n + "_exp"] = whole.reshape(s[n + "_exp"].shape)
        pool[at] = x
        got[n] = pool.reshape(s[n].shape)
    return got


def _exact_attend(case, s):
    """Sequence by sequence, in 64 bits."""
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    page, group = case["page"], case["nq"] // case["nkv"]
    for i, (n, own_keys) in enumerate(zip(_tokens(case), _lengths(case))):
        keys = case["shared"] + own_keys
        pages = s["table"][i, :-(-keys // page)].long()
        kv = []
        for name in ("k", "v"):
            x = s[name].view(torch.uint8 if s["k_exp"] is not None else torch.bfloat16)[pages].view(s[name].dtype).double()
            if s["k_exp"] is not None:
                x = x * 2.0 ** (s[name + "_exp"][pages].double() - 127.0)[..., None]
            kv.append(x.flatten(0, 1)[:keys].repeat_interleave(group, 1).permute(1, 0, 2))  # [nq, keys, d]
        z = torch.einsum("thd,hkd->htk", s["q"][i, :n].double(), kv[0]) * case["d"] ** -0.5
        for t in range(n):
            top = keys - (n - 1 - t) if case["causal"] else keys
            z[:, t, top:] = float("-inf")
            if case["window"]:
                z[:, t, :max(0, top - case["window"])] = float("-inf")
        out[i, :n] = torch.einsum("htk,hkd->thd", torch.softmax(z, 2), kv[1])
    return out.cpu().numpy()


def _exact_adjust(case, s):
    z = s["logits"].double().cpu().numpy()
    host = {n: None if s[n] is None else s[n].cpu().numpy() for n in s if n not in ("op", "logits", "out")}
    for i in range(case["batch"]):
        n, prompt = host["n_tokens"][i], host["prompt_len"][i]
        tokens = host["tokens"][i, :n]
        for r in range(case["rows"]):
            drafts = tokens[:0] if host["path"] is None else host["path"][i, :r]
            count = np.bincount(np.concatenate((tokens[prompt:], drafts)), minlength=case["vocab"])
            seen = np.unique(np.concatenate((tokens, drafts)))
            x = z[i, r]
            rep = float(host["repetition"][i])
            x[seen] = np.where(x[seen] > 0, x[seen] / rep, x[seen] * rep)
            x -= float(host["frequency"][i]) * count
            x[count > 0] -= float(host["presence"][i])
            if host["bias_id"] is not None:
                for t, value in {int(t): float(w) for t, w in zip(host["bias_id"][i], host["bias"][i]) if t >= 0}.items():
                    x[t] += value
            if host["mask"] is not None:
                bits = np.unpackbits(host["mask"][i, r].view(np.uint8), bitorder="little")[:case["vocab"]]
                x[bits == 0] = -np.inf
    return z


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    if case["op"] == "adjust":
        return _exact_adjust(case, s)
    return _exact_rows(case, s)
