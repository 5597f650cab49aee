"""What is measured of the attention calls that read a key/value cache, and of the call that shrinks it.

  sink    area_sink_attn    causal attention over a sliding window and the first tokens
  prefix  area_prefix_attn  attention of a batch that shares a long prefix, and of its own keys
  cache   area_cache_attn   causal attention over a cache that also adds up each key's weights
  evict   area_cache_evict  keeps the first, the last and the heaviest tokens of a cache

Layouts: q, o [B, H, Nq, D]; k, v [B, Hk, S, D] with S the cache's capacity and lens[b] <= S of its
tokens valid; query head h reads key head h / (H / Hk); the Nq queries of a sequence are its last
tokens.  Where `own` is false, run() computes the plain form in 32 bits with elementary operations.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}


# ---- the cases ---------------------------------------------------------------------------------

def _sink(B, H, Hk, Nq, S, D, window, sinks, dtype, low):
    return {"op": "sink", "B": B, "H": H, "Hk": Hk, "Nq": Nq, "S": S, "D": D, "window": window,
            "sinks": sinks, "dtype": dtype, "low": low}


def _prefix(B, H, Hk, Nq, P, S, D, causal, dtype, low):
    return {"op": "prefix", "B": B, "H": H, "Hk": Hk, "Nq": Nq, "P": P, "S": S, "D": D,
            "causal": causal, "dtype": dtype, "low": low}


def _cache(B, H, Hk, Nq, S, D, dtype, low):
    return {"op": "cache", "B": B, "H": H, "Hk": Hk, "Nq": Nq, "S": S, "D": D, "dtype": dtype,
            "low": low}


def _evict(B, Hk, S, D, budget, sinks, recent, So, dtype, low):
    return {"op": "evict", "B": B, "Hk": Hk, "S": S, "D": D, "budget": budget, "sinks": sinks,
            "recent": recent, "So": So, "dtype": dtype, "low": low}


def listed():
    """`low`: the shortest sequence's tokens; the batch's lengths lie evenly between it and S."""
    return [
        # one new token of two short sequences: latency
        {"name": "sink_token_small", **_sink(2, 8, 2, 1, 1000, 64, 512, 4, BF16, 301)},
        # one new token each of a serving batch, each with a window of its long cache
        {"name": "sink_token_batch", **_sink(64, 32, 8, 1, 16384, 128, 4096, 4, BF16, 3000)},
        # a prompt whose 512 text tokens stay visible while the window moves over 8192 tokens
        {"name": "sink_prompt", **_sink(1, 24, 24, 8192, 8192, 128, 2048, 512, BF16, 8192)},
        # the same in 32 bits, odd sizes, two sequences, the shorter one padded in front
        {"name": "sink_prompt_f32", **_sink(2, 6, 2, 1531, 1531, 64, 301, 7, F32, 1200)},
        # one new token of four answers to one short prompt
        {"name": "prefix_token_small", **_prefix(4, 8, 8, 1, 700, 130, 64, True, BF16, 1)},
        # one new token of 64 samples that share a long prompt
        {"name": "prefix_token_batch", **_prefix(64, 32, 8, 1, 32768, 512, 128, True, BF16, 40)},
        # four images of one prompt: each attends to the shared text and to itself, not causal
        {"name": "prefix_images", **_prefix(4, 24, 24, 4096, 512, 4096, 128, False, BF16, 4096)},
        # a few proposed tokens each, in 32 bits
        {"name": "prefix_tokens_f32", **_prefix(3, 6, 2, 5, 1999, 77, 128, True, F32, 9)},
        # one new token of a short cache in 32 bits
        {"name": "cache_token_small", **_cache(1, 8, 2, 1, 513, 64, F32, 513)},
        # one new token each of a serving batch
        {"name": "cache_token_batch", **_cache(32, 32, 8, 1, 8192, 128, BF16, 2000)},
        # a short cache back to its budget
        {"name": "evict_small", **_evict(1, 2, 600, 64, 250, 4, 64, 600, F32, 600)},
        # a serving batch's caches to half their size
        {"name": "evict_batch", **_evict(32, 8, 8192, 128, 4096, 4, 1024, 4096, BF16, 5000)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(8, 8), (8, 2), (24, 24), (32, 8), (6, 2), (16, 1), (5, 5), (12, 4)])


def draw(rng):
    op = rng.choice(["sink", "sink", "prefix", "prefix", "cache", "evict"])
    dtype, D = rng.choice([BF16, BF16, BF16, F32]), rng.choice([64, 128])
    H, Hk = _heads(rng)
    # tokens of keys and values that a call holds, and scores that it has
    held = int(1.0e9) // (2 * Hk * D * (2 if dtype == BF16 else 4))
    if op == "evict":
        S = _log(rng, 200, min(40000, held))
        B = max(1, min(_log(rng, 1, 64), held // S))
        budget = max(8, int(S * rng.uniform(0.1, 0.9)))
        sinks = rng.choice([0, 1, 4, min(64, budget // 4)])
        recent = int((budget - sinks) * rng.choice([0.0, 0.1, 0.5, 0.9]))
        return _evict(B, Hk, S, D, budget, sinks, recent, rng.choice([budget, S]), dtype,
                      int(S * rng.uniform(0.05, 1)))
    many = rng.random() < 0.4
    if many:  # a prompt or a chunk of one
        Nq, B, most = _log(rng, 40, 4096), rng.randint(1, 3), 1.5e9
    else:     # serving: one token or a few proposed ones
        Nq, B, most = rng.choice([1, 1, 1, 2, 3, 5, 8]), _log(rng, 1, 64), 0.25e9
    Nq = min(Nq, 256) if op == "cache" else Nq
    P = _log(rng, 100, 30000) if op == "prefix" else 0
    S = _log(rng, 16, 4000) if op == "prefix" else _log(rng, 100, 60000)
    P, S = min(P, held // 2, int(most / (H * Nq)) // 2), min(S, held // 2, int(most / (H * Nq)) // 2)
    P, S = max(P, 1 if op == "prefix" else 0), max(S, Nq)
    B = max(1, min(B, (held - P) // S, int(most / (H * Nq * (P + S)))))
    low = int(S * rng.uniform(0.6, 1)) if many else rng.randint(0, S)
    if op == "prefix":
        return _prefix(B, H, Hk, Nq, P, S, D, rng.random() < 0.7, dtype, low)
    if op == "cache":
        return _cache(B, H, Hk, Nq, S, D, dtype, low)
    return _sink(B, H, Hk, Nq, S, D, _log(rng, 1, S), rng.choice([0, 1, 4, 4, 77, 512]), dtype, low)


# ---- inputs ------------------------------------------------------------------------------------

def _lens(case):
    """The sequences' lengths: evenly between `low` and S."""
    B, S, low = case["B"], case["S"], case["low"]
    return [S - (S - low) * b // max(1, B - 1) for b in range(B)]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = _TYPES[case["dtype"]]
    B, S, D, Hk = case["B"], case["S"], case["D"], case["Hk"]

    def rows(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=t)

    order = torch.randperm(B, generator=g, device=dev)
    lens = torch.tensor(_lens(case), dtype=torch.int32, device=dev)[order].contiguous()
    st = {"case": case, "lens": lens, "k": rows(B, Hk, S, D), "v": rows(B, Hk, S, D)}
    if case["op"] == "evict":
        # sums of weights: a few heavy keys, many light ones, and equal values among the lightest
        u = torch.rand(B, Hk, S, generator=g, device=dev)
        st["acc"] = torch.floor(u.pow(-0.7) * 64 - 63.5).clamp_(min=0) / 64 + \
            (u < 0.5) * torch.rand(B, Hk, S, generator=g, device=dev)
        So = case["So"]
        st["ko"] = torch.zeros(B, Hk, So, D, dtype=t, device=dev)
        st["vo"] = torch.zeros(B, Hk, So, D, dtype=t, device=dev)
        return st
    H, Nq = case["H"], case["Nq"]
    st["q"] = rows(B, H, Nq, D) * 1.5
    if case["op"] == "prefix":
        st["kp"], st["vp"] = rows(Hk, case["P"], D), rows(Hk, case["P"], D)
    if case["op"] == "cache":
        st["acc"] = torch.rand(B, Hk, S, generator=g, device=dev)
    return st


# ---- the calls and their plain forms -----------------------------------------------------------

def run(state):
    if own:
        return _OWN[state["case"]["op"]](state, state["case"])
    return _PLAIN[state["case"]["op"]](state, state["case"])


def _scores(q, k, Hk, D):
    """q [B, H, Nq, D] times k [B or 1, Hk, n, D] over sqrt(D): [B, Hk, G, Nq, n]."""
    B, H, Nq, _ = q.shape
    q = q.float().reshape(B, Hk, H // Hk * Nq, D)
    s = torch.matmul(q, k.float().transpose(-1, -2)).mul_(D ** -0.5)
    return s.view(B, Hk, H // Hk, Nq, k.shape[2])


def _weights(s, mask):
    """Softmax over the last axis of what `mask` leaves; a row that it leaves nothing has no weights."""
    s = s.masked_fill_(~mask, float("-inf"))
    top = s.amax(-1, keepdim=True)
    s = s.sub_(torch.where(top > float("-inf"), top, torch.zeros_like(top))).exp_()
    total = s.sum(-1, keepdim=True)
    return s.div_(torch.where(total > 0, total, torch.ones_like(total)))


def _values(w, v, like):
    """w [B, Hk, G, Nq, n] times v [B, Hk, n, D], in the type and layout of q."""
    B, Hk, G, Nq, n = w.shape
    o = torch.matmul(w.view(B, Hk, G * Nq, n), v.float())
    return o.view(like.shape).to(like.dtype)


def _own_keys(v, lens):
    """v with zeros behind each sequence's last token."""
    at = torch.arange(v.shape[2], device=v.device)
    return v.masked_fill((at >= lens[:, None])[:, None, :, None], 0)


def _positions(lens, Nq):
    return lens[:, None] - Nq + torch.arange(Nq, device=lens.device)      # [B, Nq]


def _plain_sink(st, c):
    at = torch.arange(c["S"], device=st["q"].device)
    p = _positions(st["lens"], c["Nq"])[:, :, None]                       # [B, Nq, 1]
    mask = (at <= p) & ((at < c["sinks"]) | (at > p - c["window"]))       # [B, Nq, S]
    w = _weights(_scores(st["q"], st["k"], c["Hk"], c["D"]), mask[:, None, None])
    return {"o": _values(w, _own_keys(st["v"], st["lens"]), st["q"])}


def _plain_prefix(st, c):
    at = torch.arange(c["S"], device=st["q"].device)
    p = _positions(st["lens"], c["Nq"])[:, :, None]
    if c["causal"]:
        mine, shared = at <= p, p >= 0
    else:
        mine, shared = at < st["lens"][:, None, None].expand_as(p), torch.ones_like(p, dtype=torch.bool)
    mask = torch.cat([shared.expand(-1, -1, c["P"]), mine], -1)
    k, v = st["k"], _own_keys(st["v"], st["lens"])
    s = torch.cat([_scores(st["q"], st["kp"][None], c["Hk"], c["D"]),
                   _scores(st["q"], k, c["Hk"], c["D"])], -1)
    w = _weights(s, mask[:, None, None])
    v = torch.cat([st["vp"].expand(c["B"], -1, -1, -1), v], 2)
    return {"o": _values(w, v, st["q"])}


def _plain_cache(st, c):
    at = torch.arange(c["S"], device=st["q"].device)
    mask = at <= _positions(st["lens"], c["Nq"])[:, :, None]
    w = _weights(_scores(st["q"], st["k"], c["Hk"], c["D"]), mask[:, None, None])
    return {"o": _values(w, _own_keys(st["v"], st["lens"]), st["q"]), "acc": st["acc"] + w.sum((2, 3))}


def _plain_evict(st, c):
    B, Hk, S, So, budget = c["B"], c["Hk"], c["S"], c["So"], c["budget"]
    acc, n = st["acc"], st["lens"][:, None, None]                          # n [B, 1, 1]
    at = torch.arange(S, device=acc.device)
    always = (n <= budget) | (at < c["sinks"]) | (at >= n - c["recent"])
    free = ~always & (at < n)
    key = torch.where(free, acc, float("-inf"))
    rank = key.argsort(dim=-1, descending=True, stable=True).argsort(dim=-1)
    keep = (at < n) & (always | (free & (rank < budget - c["sinks"] - c["recent"])))
    idx = torch.where(keep, at, S).sort(-1).values
    idx = torch.nn.functional.pad(idx, (0, max(0, So - S)), value=S)[..., :So]
    had = idx < S
    src = torch.where(had, idx, 0)
    rows = src[..., None].expand(-1, -1, -1, c["D"])
    hole = had[..., None]
    return {"k": torch.where(hole, st["k"].gather(2, rows), st["ko"]),
            "v": torch.where(hole, st["v"].gather(2, rows), st["vo"]),
            "acc": torch.where(had, acc.gather(2, src), 0.0),
            "idx": torch.where(had, idx, -1).int(),
            "lens": st["lens"].clamp(max=budget)}


_PLAIN = {"sink": _plain_sink, "prefix": _plain_prefix, "cache": _plain_cache, "evict": _plain_evict}


def _kept(st, name, make):
    """A workspace or output buffer that the program keeps from call to call."""
    if name not in st:
        st[name] = make()
    return st[name]


def _workspace(st, nbytes):
    return _kept(st, "ws", lambda: torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda"))


def _own_sink(st, c):
    import step_adaptive_sparse_b200 as area
    d = area.AREA_DTYPE_BF16 if c["dtype"] == BF16 else area.AREA_DTYPE_F32
    size = [c[n] for n in ("B", "H", "Hk", "Nq", "S", "D", "window", "sinks")]
    nb = area.area_sink_attn_ws_bytes(*size, d)
    ws, o = _workspace(st, nb), torch.empty_like(st["q"])
    area.area_sink_attn(st["q"], st["k"], st["v"], st["lens"], o, ws, nb, *size, c["D"] ** -0.5, d,
                        torch.cuda.current_stream())
    return {"o": o}


def _own_prefix(st, c):
    import step_adaptive_sparse_b200 as area
    d = area.AREA_DTYPE_BF16 if c["dtype"] == BF16 else area.AREA_DTYPE_F32
    size = [c[n] for n in ("B", "H", "Hk", "Nq", "P", "S", "D")]
    nb = area.area_prefix_attn_ws_bytes(*size, d)
    ws, o = _workspace(st, nb), torch.empty_like(st["q"])
    area.area_prefix_attn(st["q"], st["kp"], st["vp"], st["k"], st["v"], st["lens"], o, ws, nb,
                          *size, int(c["causal"]), c["D"] ** -0.5, d, torch.cuda.current_stream())
    return {"o": o}


def _own_cache(st, c):
    import step_adaptive_sparse_b200 as area
    d = area.AREA_DTYPE_BF16 if c["dtype"] == BF16 else area.AREA_DTYPE_F32
    size = [c[n] for n in ("B", "H", "Hk", "Nq", "S", "D")]
    nb = area.area_cache_attn_ws_bytes(*size, d)
    ws, o, acc = _workspace(st, nb), torch.empty_like(st["q"]), torch.empty_like(st["acc"])
    area.area_cache_attn(st["q"], st["k"], st["v"], st["lens"], st["acc"], o, acc, ws, nb, *size,
                         c["D"] ** -0.5, d, torch.cuda.current_stream())
    return {"o": o, "acc": acc}


def _own_evict(st, c):
    import step_adaptive_sparse_b200 as area
    d = area.AREA_DTYPE_BF16 if c["dtype"] == BF16 else area.AREA_DTYPE_F32
    B, Hk, So = c["B"], c["Hk"], c["So"]
    acc = torch.empty(B, Hk, So, device="cuda")
    idx = torch.empty(B, Hk, So, dtype=torch.int32, device="cuda")
    lens = torch.empty_like(st["lens"])
    area.area_cache_evict(st["k"], st["v"], st["acc"], st["lens"], st["ko"], st["vo"], acc, lens, idx,
                          B, Hk, c["S"], So, c["D"], c["budget"], c["sinks"], c["recent"], d,
                          torch.cuda.current_stream())
    return {"k": st["ko"], "v": st["vo"], "acc": acc, "idx": idx, "lens": lens}


_OWN = {"sink": _own_sink, "prefix": _own_prefix, "cache": _own_cache, "evict": _own_evict}


# ---- what a pass cannot do without -------------------------------------------------------------

def _up_to(n, limit):
    """Sum of min(i, limit) over i = 1 .. n."""
    m = min(n, limit)
    return m * (m + 1) // 2 + (n - m) * limit


def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    B, Hk, S, D = case["B"], case["Hk"], case["S"], case["D"]
    lens = _lens(case)
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        read = sum(lens)
        return {"bytes": Hk * (kept * 4 * D * e + 4 * read + B * case["So"] * 8), "flops": Hk * read}
    H, Nq = case["H"], case["Nq"]
    io = 2 * B * H * Nq * D * e
    if case["op"] == "sink":
        pairs = keys = 0
        for n in lens:
            first = max(1, n - Nq + 1)      # keys of the first query of this sequence
            m, s = case["window"], case["sinks"]
            # a query that sees i keys in all attends to min(i, m) of the window and to the
            # sinks before it, min(s, max(0, i - m))
            pairs += _up_to(n, m) - _up_to(first - 1, m)
            pairs += _up_to(max(0, n - m), s) - _up_to(max(0, first - 1 - m), s)
            lo = max(0, first - m)
            keys += n - lo + min(s, lo)
        return {"bytes": io + keys * Hk * 2 * D * e, "flops": 4 * D * H * pairs}
    if case["op"] == "prefix":
        if case["causal"]:
            pairs = sum(_up_to(n, n) - _up_to(max(0, n - Nq), n) + min(Nq, n) * case["P"] for n in lens)
        else:
            pairs = sum(Nq * (n + case["P"]) for n in lens)
        return {"bytes": io + (sum(lens) + case["P"]) * Hk * 2 * D * e, "flops": 4 * D * H * pairs}
    pairs = sum(_up_to(n, n) - _up_to(max(0, n - Nq), n) for n in lens)
    return {"bytes": io + sum(lens) * Hk * 2 * D * e + 2 * B * Hk * S * 4, "flops": 4 * D * H * pairs}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(st, case)
    B, H, Hk, Nq, D = (case[n] for n in ("B", "H", "Hk", "Nq", "D"))
    if 4 * D * B * H * Nq * (case["S"] + case.get("P", 0)) > 2e13:
        return None
    o = torch.zeros(B, H, Nq, D, dtype=torch.float64, device="cuda")
    acc = st["acc"].double() if case["op"] == "cache" else None
    step = max(1, (1 << 27) // (case["S"] + case.get("P", 0)))
    for b, n in enumerate(st["lens"].tolist()):
        for h in range(H):
            hk = h * Hk // H
            keys, vals = st["k"][b, hk, :n].double(), st["v"][b, hk, :n].double()
            if case["op"] == "prefix":
                keys = torch.cat([st["kp"][hk].double(), keys])
                vals = torch.cat([st["vp"][hk].double(), vals])
            own_at = torch.arange(keys.shape[0], device="cuda") - (keys.shape[0] - n)
            for i in range(0, Nq, step):
                pos = n - Nq + torch.arange(i, min(Nq, i + step), device="cuda")[:, None]
                sees = own_at <= pos
                if case["op"] == "sink":
                    sees &= (own_at < case["sinks"]) | (pos - own_at < case["window"])
                if case["op"] == "prefix":
                    sees = (sees & (pos >= 0)) if case["causal"] else torch.ones_like(sees)
                x = (st["q"][b, h, i:i + step].double() @ keys.T) / math.sqrt(D)
                x = torch.where(sees, x, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
                w = torch.softmax(x, -1).nan_to_num(0.0)                   # NaN: a row that sees nothing
                o[b, h, i:i + step] = w @ vals
                if acc is not None:
                    acc[b, hk, :n] += w.sum(0)
    return {"o": o, "acc": acc} if acc is not None else {"o": o}


def _exact_evict(st, c):
    B, Hk, So, budget, sinks, recent = (c[n] for n in ("B", "Hk", "So", "budget", "sinks", "recent"))
    acc = st["acc"].cpu()
    out = torch.zeros(B, Hk, So, dtype=torch.float64)
    k = torch.zeros(B, Hk, So, c["D"], dtype=torch.float64, device="cuda")
    v = torch.zeros_like(k)
    for b, n in enumerate(st["lens"].tolist()):
        for h in range(Hk):
            kept = torch.arange(n)
            if n > budget:
                free = acc[b, h, sinks:n - recent]
                best = torch.sort(free, descending=True, stable=True).indices[:budget - sinks - recent]
                kept = torch.cat([kept[:sinks], best.sort().values + sinks, kept[n - recent:]])
            m = len(kept)
            out[b, h, :m] = acc[b, h, kept].double()
            k[b, h, :m] = st["k"][b, h, kept.cuda()].double()
            v[b, h, :m] = st["v"][b, h, kept.cuda()].double()
    return {"k": k, "v": v, "acc": out, "idx": None, "lens": None}
