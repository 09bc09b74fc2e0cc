"""Workloads of the library's stand-alone operators: the product with 4-bit weights, and the operators that turn a
target's logits into tokens (sampling, the truncated distribution, sampled verification of a draft).

Each operator has a plain form in elementary torch operations (``own`` false) and the library's call (``own`` true) on
the same inputs; ``exact`` gives the 64-bit result from the definition.

Definitions
  4-bit weights: byte j of a row of ``codes`` holds element 2j in its low and 2j + 1 in its high nibble; the weight is
    (nibble - 8) * scale[row][element // group].
  Truncation of a row of logits z at temperature T: T <= 0 leaves the largest logit alone; otherwise the tokens are
    ordered by logit (equal logits: smaller id first), the first top_k stay, of these the shortest prefix that holds
    top_p of their mass, of these the ones with at least min_p of the largest one's mass; the mass of a token is
    exp((z - max z) / T).  Tokens at -inf have no mass and never stay.
  A draw with number u takes the first token, in id order, whose cumulative mass exceeds u times the total.
  Verification: draft i is accepted while u_accept[i] is below the probability of its token in row i; the token after
    the accepted prefix is drawn from its row, without the rejected draft's token if there is one.
"""

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------------------------------------- cases

def _linear(name, out_features, in_features, rows, group, out):
    c = {"op": "linear_w4", "out_features": out_features, "in_features": in_features, "rows": rows, "group": group,
         "out": out}
    return dict(c, name=name) if name else c


def _logits(op, name, batch, rows, vocab, dtype, shape, settings, masked=False):
    c = {"op": op, "batch": batch, "rows": rows, "vocab": vocab, "dtype": dtype, "shape": shape, "settings": settings,
         "masked": masked}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the smallest projection of the small test model, one token: latency alone
        _linear("linear_small_1", 704, 256, 1, 32, "f32"),
        # the readout of one token of the 8B-shaped target (plain decoding between two drafts)
        _linear("linear_lm_head_1", 151936, 4096, 1, 128, "f32"),
        # the same readout of a verify batch: the anchor and seven drafts
        _linear("linear_lm_head_8", 151936, 4096, 8, 64, "f32"),
        # the down projection of the 27B-shaped draft at batch 8 x block 16
        _linear("linear_down_128", 5120, 17408, 128, 128, "bf16"),
        # the first anchor of one request: the settings the DFlash 2 evaluations quote
        _logits("sample", "sample_1", 1, 1, 151936, "f32", "peaked", "evaluation"),
        # one token of each of 64 requests with their own settings, bf16 logits as a readout stores them
        _logits("sample", "sample_64_mixed", 64, 1, 151936, "bf16", "peaked", "mixed"),
        # temperature alone over a wide, flat distribution, an odd vocabulary
        _logits("sample", "sample_200_plain", 200, 1, 50257, "f32", "flat", "temperature"),
        # the distribution rows of one verify batch, for verify_sampled
        _logits("target_probs", "probs_8", 1, 8, 151936, "f32", "peaked", "evaluation"),
        # the same of 16 requests, a nucleus over a flat distribution (tens of thousands of tokens stay)
        _logits("target_probs", "probs_128_nucleus", 16, 8, 151936, "bf16", "flat", "nucleus"),
        # the verify batch of the small test model, a grammar mask over part of the vocabulary
        _logits("verify", "verify_small_masked", 3, 8, 1000, "f32", "peaked", "evaluation", True),
        # the verify batch of one request at the 8B shape
        _logits("verify", "verify_8", 1, 8, 151936, "f32", "peaked", "evaluation"),
        # 32 requests with their own settings and draft counts
        _logits("verify", "verify_256_mixed", 32, 8, 151936, "bf16", "peaked", "mixed"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    if rng.random() < 0.34:
        group = rng.choice((32, 64, 128))
        k = group * _log(rng, 2, 17408 // group)
        m = _log(rng, 100, min(151936, 600_000_000 // k))
        rows = _log(rng, 1, max(1, min(256, 12_000_000_000 // (m * k))))
        return _linear(None, m, k, rows, group, rng.choice(("f32", "bf16")))
    op = rng.choice(("sample", "target_probs", "verify"))
    vocab = _log(rng, 500, 151936)
    most = 256 * 151936 // vocab
    rows = 1 if op == "sample" else rng.randint(2, 16)
    batch = _log(rng, 1, max(1, min(256, most) // rows))
    return _logits(op, None, batch, rows, vocab, rng.choice(("f32", "bf16")), rng.choice(("peaked", "flat")),
                   rng.choice(("evaluation", "mixed", "temperature", "nucleus")), rng.random() < 0.25)


def work(case):
    if case["op"] == "linear_w4":
        m, k, n = case["out_features"], case["in_features"], case["rows"]
        out = 4 if case["out"] == "f32" else 2
        return {"bytes": m * k / 2 + 2 * m * k / case["group"] + 2 * n * k + out * n * m, "flops": 2.0 * m * n * k}
    n, v = case["batch"] * case["rows"], case["vocab"]
    size = 4 if case["dtype"] == "f32" else 2
    bytes_ = n * v * size + 32.0 * n
    if case["op"] == "target_probs":
        bytes_ += 4.0 * n * v
    return {"bytes": bytes_, "flops": 4.0 * n * v}  # a difference, a product, an exponential and a sum each


# --------------------------------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _prepare_linear(case, g):
    m, k, n, group = case["out_features"], case["in_features"], case["rows"], case["group"]
    w = torch.randn((m, k // group, group), generator=g, device="cuda") * 0.02
    scale = (w.abs().amax(2) / 7).to(torch.bfloat16)
    q = (w / scale.float()[:, :, None]).round_().clamp_(-8, 7).add_(8).to(torch.uint8).reshape(m, k)
    x = torch.randn((n, k), generator=g, device="cuda").to(torch.bfloat16)
    return {"codes": q[:, 0::2] | (q[:, 1::2] << 4), "scale": scale, "x": x,
            "out": torch.empty((n, m), dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device="cuda")}


def _settings(kind, n, g):
    """Per-request temperature, top_k, top_p and min_p; None where no request uses the filter."""
    uniform = lambda lo, hi: torch.rand((n,), generator=g, device="cuda") * (hi - lo) + lo  # noqa: E731
    full = lambda v, t: torch.full((n,), v, dtype=t, device="cuda")  # noqa: E731
    if kind == "evaluation":
        return full(1.0, torch.float32), full(20, torch.int32), full(0.95, torch.float32), None
    if kind == "nucleus":
        return full(1.0, torch.float32), None, full(0.9, torch.float32), None
    if kind == "temperature":
        return uniform(0.7, 1.1), None, None, None
    chosen = torch.rand((4, n), generator=g, device="cuda")
    temperature = torch.where(chosen[0] < 0.125, torch.zeros((n,), device="cuda"), uniform(0.3, 1.3))
    top_k = torch.where(chosen[1] < 0.3, torch.zeros((n,), device="cuda"), uniform(1, 100)).to(torch.int32)
    top_p = torch.where(chosen[2] < 0.3, torch.ones((n,), device="cuda"), uniform(0.7, 1.0))
    min_p = torch.where(chosen[3] < 0.5, torch.zeros((n,), device="cuda"), uniform(0.02, 0.1))
    return temperature, top_k, top_p, min_p


def _prepare_logits(case, g):
    b, r, v = case["batch"], case["rows"], case["vocab"]
    z = torch.randn((b, r, v), generator=g, device="cuda")
    if case["shape"] == "peaked":  # a head of likely tokens with falling logits over a bulk, as trained models give
        n = min(64, v // 4)
        ids = torch.argsort(torch.rand((b * r, 4 * n), generator=g, device="cuda"), 1)[:, :n].reshape(b, r, n)
        ids = (ids * (v // (4 * n))).to(torch.int64)
        rank = torch.arange(1, n + 1, device="cuda", dtype=torch.float32)
        head = 15 - 1.2 * rank.log() + 0.3 * torch.randn((b, r, n), generator=g, device="cuda")
        z = (z * 1.2).scatter_(2, ids, head)
    if case["masked"]:
        z = z.masked_fill_(torch.rand((b, r, v), generator=g, device="cuda") < 0.25, float("-inf"))
    s = {"logits": z if case["dtype"] == "f32" else z.to(torch.bfloat16)}
    s["settings"] = _settings(case["settings"], b, g)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    if case["op"] == "sample":
        s["u"] = torch.rand((b,), generator=g, device="cuda")
        s["token"], s["prob"] = torch.empty((b,), **i32), torch.empty((b,), device="cuda")
    elif case["op"] == "target_probs":
        s["prob"] = torch.empty((b, r, v), device="cuda")
    else:
        # drafts that mostly agree with the target, as a trained draft's do; some requests keep fewer of them
        likely = torch.topk(s["logits"][:, :r - 1].float(), min(8, v), dim=2).indices
        other = torch.randint(0, likely.shape[2], (b, r - 1, 1), generator=g, device="cuda")
        other = torch.where(torch.rand((b, r - 1, 1), generator=g, device="cuda") < 0.75, 0, other)
        s["path"] = torch.gather(likely, 2, other).squeeze(2).to(torch.int32).contiguous()
        s["n_draft"] = torch.randint(0, r, (b,), generator=g, **i32) if case["settings"] == "mixed" else None
        s["u_accept"] = torch.rand((b, r - 1), generator=g, device="cuda")
        s["u"] = torch.rand((b,), generator=g, device="cuda")
        s["accept_len"], s["n_out"], s["next_anchor"] = (torch.empty((b,), **i32) for _ in range(3))
        s["out_tok"] = torch.empty((b, r), **i32)
        s["workspace"] = torch.zeros((4096 + 64 * b * r,), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    g = _generator(seed)
    s = _prepare_linear(case, g) if case["op"] == "linear_w4" else _prepare_logits(case, g)
    return dict(s, op=case["op"], group=case.get("group"))


# ----------------------------------------------------------------------------------------------------- plain forms

def _plain_linear(s):
    codes, scale, group = s["codes"], s["scale"], s["group"]
    m, half = codes.shape
    q = torch.stack((codes & 15, codes >> 4), 2).reshape(m, 2 * half // group, group).float() - 8
    w = (q * scale.float()[:, :, None]).reshape(m, 2 * half)
    return (s["x"].float() @ w.t()).to(s["out"].dtype)


def _masses(logits, settings):
    """[batch, rows, vocab] logits -> the masses of the tokens that stay, in id order, in 64 bits."""
    z = logits.float()
    temperature, top_k, top_p, min_p = (None if p is None else p[:, None, None] for p in settings)
    zs, ids = torch.sort(z, dim=2, descending=True, stable=True)
    place = torch.arange(z.shape[2], device=z.device)
    t = torch.ones_like(zs[:, :1, :1]) if temperature is None else temperature
    e = torch.where(zs == zs[..., :1], 0.0, (zs.double() - zs[..., :1].double()) / t.double()).exp()
    e = e * (zs > float("-inf"))
    if top_k is not None:
        e = e * ((place < top_k) | (top_k <= 0))
    if top_p is not None:
        c = e.cumsum(2)
        e = e * ((c - e < top_p.double() * c[..., -1:]) | (place == 0) | (top_p >= 1))
    if min_p is not None:
        e = e * (e >= min_p.double())
    e = torch.where(t > 0, e, ((place == 0) & (zs > float("-inf"))).double())
    return torch.zeros_like(e).scatter_(2, ids, e)


def _draw(mass, u):
    """First id whose cumulative mass exceeds u times the total; mass [n, vocab], u [n]."""
    c = mass.cumsum(1)
    return (c <= u.double()[:, None] * c[:, -1:]).sum(1)


def _plain_sample(s):
    mass = _masses(s["logits"], s["settings"])[:, 0]
    token = _draw(mass, s["u"])
    prob = mass.gather(1, token[:, None]).squeeze(1) / mass.sum(1)
    return {"token": token.to(torch.int32), "prob": prob.float()}


def _plain_probs(s):
    mass = _masses(s["logits"], s["settings"])
    return (mass / mass.sum(2, keepdim=True)).float()


def _plain_verify(s):
    b, rows, v = s["logits"].shape
    mass = _masses(s["logits"], s["settings"])
    path = s["path"].to(torch.int64)
    place = torch.arange(rows - 1, device=path.device)
    n = torch.full((b,), rows - 1, device=path.device) if s["n_draft"] is None else s["n_draft"]
    px = mass[:, :-1].gather(2, path[:, :, None]).squeeze(2)
    ok = (s["u_accept"].double() * mass[:, :-1].sum(2) < px) & (place < n[:, None])
    a = ok.to(torch.int64).cumprod(1).sum(1)
    row = mass.gather(1, a[:, None, None].expand(b, 1, v)).squeeze(1)
    last = path.gather(1, a.clamp(max=rows - 2)[:, None])
    rejected = (a < n)[:, None] & (torch.arange(v, device=path.device) == last)
    token = _draw(row.masked_fill(rejected, 0.0), s["u"]).to(torch.int32)
    slots = torch.arange(rows, device=path.device)
    out = torch.cat((s["path"], torch.full((b, 1), -1, dtype=torch.int32, device=path.device)), 1)
    out = torch.where(slots < a[:, None], out, torch.where(slots == a[:, None], token[:, None], -1))
    a = a.to(torch.int32)
    return {"accept_len": a, "out_tok": out.to(torch.int32), "n_out": a + 1, "next_anchor": token}


# ------------------------------------------------------------------------------------------------- the library's

def _library():
    from block_speculative_decoding_dflash2_gb300 import binding
    return binding


def _own(s):
    lib = _library()
    if s["op"] == "linear_w4":
        lib.dflash2_linear_w4(s["codes"], s["scale"], s["group"], s["x"], s["out"])
        return s["out"]
    if s["op"] == "sample":
        lib.dflash2_sample(s["logits"][:, 0], *s["settings"], s["u"], s["token"], s["prob"])
        return {"token": s["token"], "prob": s["prob"]}
    if s["op"] == "target_probs":
        lib.dflash2_target_probs(s["logits"], *s["settings"], s["prob"])
        return s["prob"]
    lib.dflash2_verify_logits(s["path"], s["n_draft"], s["logits"], *s["settings"], s["u_accept"], s["u"],
                              s["accept_len"], s["out_tok"], s["n_out"], s["next_anchor"], s["workspace"])
    return {k: s[k] for k in ("accept_len", "out_tok", "n_out", "next_anchor")}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "linear_w4":
        return _plain_linear(state)
    if state["op"] == "sample":
        return _plain_sample(state)
    if state["op"] == "target_probs":
        return _plain_probs(state)
    return _plain_verify(state)


# ------------------------------------------------------------------------------------------------- 64-bit results

def _exact_linear(s):
    """Row blocks of the product in 64 bits."""
    x, group = s["x"].double(), s["group"]
    m, half = s["codes"].shape
    out = torch.empty((x.shape[0], m), dtype=torch.float64, device="cuda")
    for lo in range(0, m, 8192):
        codes = s["codes"][lo:lo + 8192].to(torch.int32)
        w = torch.empty((codes.shape[0], 2 * half), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = codes % 16 - 8, codes // 16 - 8
        w *= s["scale"][lo:lo + 8192].double().repeat_interleave(group, 1)
        out[:, lo:lo + 8192] = x @ w.t()
    return out.cpu().numpy()


def _exact_row(z, t, k, p, m):
    """Probabilities of one row of float64 logits, by the definition."""
    v = len(z)
    prob = np.zeros(v)
    if not np.any(z > -np.inf):
        return prob
    if t is not None and t <= 0:
        prob[int(np.argmax(z))] = 1.0
        return prob
    order = np.lexsort((np.arange(v), -z))
    order = order[z[order] > -np.inf]
    if k is not None and k > 0:
        order = order[:int(k)]
    mass = np.exp((z[order] - z[order[0]]) / (1.0 if t is None else t))
    if p is not None and p < 1:
        total = np.cumsum(mass)
        stay = 1 + int(np.searchsorted(total, p * total[-1], side="left"))
        order, mass = order[:max(1, stay)], mass[:max(1, stay)]
    if m is not None:
        order, mass = order[mass >= m], mass[mass >= m]
    prob[order] = mass / mass.sum()
    return prob


def _exact_token(prob, u):
    c = np.cumsum(prob)
    return int(np.searchsorted(c, u * c[-1], side="right"))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear_w4":
        return _exact_linear(s)
    z = s["logits"].double().cpu().numpy()
    settings = [None if p is None else p.double().cpu().numpy() for p in s["settings"]]
    at = lambda i: [None if p is None else p[i].item() for p in settings]  # noqa: E731
    b, rows, _ = z.shape
    if case["op"] == "target_probs":
        return np.stack([np.stack([_exact_row(z[i, j], *at(i)) for j in range(rows)]) for i in range(b)])
    u = s["u"].double().cpu().numpy()
    if case["op"] == "sample":
        token, prob = np.empty(b, np.int32), np.empty(b)
        for i in range(b):
            p = _exact_row(z[i, 0], *at(i))
            token[i] = _exact_token(p, u[i])
            prob[i] = p[token[i]]
        return {"token": token, "prob": prob}
    path, ua = s["path"].cpu().numpy(), s["u_accept"].double().cpu().numpy()
    kept = np.full(b, rows - 1) if s["n_draft"] is None else s["n_draft"].cpu().numpy()
    accept, out, nxt = np.zeros(b, np.int32), np.full((b, rows), -1, np.int32), np.zeros(b, np.int32)
    for i in range(b):
        a = 0
        p = _exact_row(z[i, 0], *at(i))
        while a < kept[i] and ua[i, a] < p[path[i, a]]:
            out[i, a] = path[i, a]
            a += 1
            p = _exact_row(z[i, a], *at(i))
        if a < kept[i]:
            p[path[i, a]] = 0.0
        accept[i], nxt[i] = a, _exact_token(p, u[i])
        out[i, a] = nxt[i]
    return {"accept_len": accept, "out_tok": out, "n_out": accept + 1, "next_anchor": nxt}
