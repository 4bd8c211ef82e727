"""Differential attention over the 8-bit paged cache, the weight that its keys
gather, and eviction of the keys that gathered least, case by case. `own` false
computes each in elementary torch operations; `own` true makes the calls a user
makes of the framework.

Notation of the cases: `n` sequences, `hkv` KV heads of `g` query heads each,
head dimension `d`, pages of `page` tokens; cached lengths spread over
[len_lo, len_hi] and rows a sequence over [new_lo, new_hi] (its last tokens, of
len + rows in all; 0 rows where nothing is attended), the same for every seed.
A page and KV head has one float32 scale for K and one for V; a stored value is
code * scale.
"""

import math

import torch

own = False

TOP = {"int8": 127.0, "e4m3": 448.0}
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases

def _rows(op, name, code, n, len_lo, len_hi, new_lo, new_hi, hkv, g, d, page, cap=0.0, slopes=False, window=0,
          prefix=0, docs=False, **more):
    c = {"op": op, "code": code, "n": n, "len_lo": len_lo, "len_hi": len_hi, "new_lo": new_lo, "new_hi": new_hi,
         "hkv": hkv, "g": g, "d": d, "page": page, "cap": cap, "slopes": slopes, "window": window, "prefix": prefix,
         "docs": docs, **more}
    return {"name": name, **c} if name else c


def _diff(name, *shape, norm=False, each=False, **score):
    """norm: the difference is normalised over its head; each: a factor for every row, else one a pair of heads."""
    return _rows("diff", name, *shape, norm=norm, each=each, **score)


def _weigh(name, *shape, alpha=1.0, decay=1.0, coef=False, whole=False, **score):
    """coef: rows and heads count by factors; whole: every key's weight begins at these rows, else the rows' own."""
    return _rows("weigh", name, *shape, alpha=alpha, decay=decay, coef=coef, whole=whole, **score)


def _evict(name, code, n, len_lo, len_hi, hkv, d, page, keep, above, sinks, recent, zeros):
    """zeros: the share of keys that gathered exactly nothing."""
    c = {"op": "evict", "code": code, "n": n, "len_lo": len_lo, "len_hi": len_hi, "new_lo": 0, "new_hi": 0,
         "hkv": hkv, "g": 4, "d": d, "page": page, "keep": keep, "above": above, "sinks": sinks, "recent": recent,
         "zeros": zeros}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one user's next token, the difference normalised over its head: latency
        _diff("difference, one sequence", "int8", 1, 32768, 32768, 1, 1, 8, 4, 128, 32, norm=True),
        # batched serving, lengths far apart, a factor from every token, linear distance bias
        _diff("difference, ragged batch", "e4m3", 16, 4096, 65536, 1, 1, 8, 4, 128, 16, each=True, slopes=True),
        # several drafted tokens checked at once, sliding window with a kept prefix
        _diff("difference, drafted tokens", "int8", 24, 1000, 20000, 2, 5, 4, 8, 64, 32, window=4096, prefix=100),
        # a prompt's chunk against a long context
        _diff("difference, prompt chunk", "int8", 1, 30001, 30001, 2048, 2048, 8, 4, 128, 32, norm=True, each=True),
        # ragged chunks, several documents in a sequence and rows that see nothing
        _diff("difference, ragged chunks", "e4m3", 6, 500, 8000, 60, 1500, 4, 6, 64, 16, norm=True, docs=True, cap=30.0),
        # what one user's next token gives to each key: latency
        _weigh("weights, one sequence", "int8", 1, 32768, 32768, 1, 1, 8, 4, 128, 32),
        # entmax decode of a batch, older weight fading away
        _weigh("weights, entmax batch", "e4m3", 16, 1000, 32000, 1, 1, 8, 4, 128, 16, alpha=1.5, decay=0.98),
        # all rows of a prompt's chunk, two maps of a differential attention counted together
        _weigh("weights, prompt chunk", "int8", 1, 30001, 30001, 2048, 2048, 8, 4, 128, 32, coef=True),
        # the last rows of prompts decide what is kept of each
        _weigh("weights, last rows", "e4m3", 6, 500, 32000, 64, 64, 8, 4, 128, 16, whole=True, slopes=True),
        # behind a decode step: one sequence in four is over its limit
        _evict("evict, decode step", "int8", 64, 200, 2600, 8, 128, 32, 2048, 2303, 4, 64, 0.0),
        # prompts of a batch, most keys without any weight (entmax): ties
        _evict("evict, batch of prompts", "e4m3", 16, 1000, 32000, 8, 64, 16, 1024, 1024, 4, 256, 0.7),
        # one long context down to an eighth
        _evict("evict, long context", "int8", 1, 131072, 131072, 8, 128, 32, 16384, 16384, 16, 2048, 0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["diff", "diff chunk", "weigh", "weigh chunk", "evict", "evict"])
    code, page, d = rng.choice(["int8", "e4m3"]), rng.choice([16, 32]), rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    if kind == "evict":
        n = _log(rng, 1, 64)
        hi = _log(rng, 40, min(131072, 500000 // n))
        keep = max(2, int(hi * math.exp(-rng.uniform(0.02, 3.0))))
        sinks = min(keep, rng.choice([0, 1, 4, keep // 8]))
        recent = min(keep - sinks, rng.choice([0, 1, (keep - sinks) // 3, keep]))
        return _evict(None, code, n, max(1, hi // rng.choice([1, 3, 30])), hi, hkv, d, page, keep,
                      rng.choice([keep, keep + (hi - keep) // 3]), sinks, recent, rng.choice([0.0, 0.3, 0.9]))
    score = {"cap": rng.choice([0.0, 0.0, rng.uniform(5.0, 60.0)]), "slopes": rng.random() < 0.3,
             "docs": rng.random() < 0.25, "window": rng.choice([0, 0, _log(rng, 1, 5000)]),
             "prefix": rng.choice([0, 0, _log(rng, 1, 400)])}
    if kind.endswith("chunk"):
        n = _log(rng, 1, 8)
        new = _log(rng, 6, 2000 // n)
        lo = _log(rng, 1, 4000)
        lens = (n, lo, lo + _log(rng, 1, 16000), rng.choice([1, new]), new)
        most = 4
    else:
        n = _log(rng, 1, 64)
        hi = _log(rng, 2, min(131072, 360000 // n))
        lens = (n, max(1, hi // rng.choice([1, 3, 10, 100])), hi, 1, rng.choice([1, 1, 1, 2, 4, 8]))
        most = 8
    if kind.startswith("diff"):
        return _diff(None, code, *lens, hkv, rng.choice(range(2, most + 1, 2)), d, page, norm=rng.random() < 0.5,
                     each=rng.random() < 0.5, **score)
    alpha = rng.choice([1.0, 1.25, 1.5, 2.0]) if lens[-1] == 1 else 1.0
    return _weigh(None, code, *lens, hkv, rng.randint(1, most), d, page, alpha=alpha, decay=rng.choice([1.0, 1.0, 0.9, 0.0]),
                  coef=rng.random() < 0.4, whole=rng.random() < 0.2, **score)


def _spread(n, lo, hi, turn):
    """n whole numbers over [lo, hi], far apart ones next to each other."""
    if n == 1:
        return [hi]
    a, b = math.log(lo + 1.0), math.log(hi + 1.0)
    v = [min(hi, max(lo, int(round(math.exp(a + (b - a) * i / (n - 1)) - 1.0)) - (i * 7) % 3)) for i in range(n)]
    step = next(s for s in range(turn, turn + n + 2) if math.gcd(s, n) == 1)
    return [v[(i * step) % n] for i in range(n)]


def _lengths(case):
    """(cached tokens in front, rows) of each sequence."""
    return (_spread(case["n"], case["len_lo"], case["len_hi"], 5),
            _spread(case["n"], case["new_lo"], case["new_hi"], 3))


def _doc(old, i):
    """First key that row i sees: every 97 rows another document begins, and every 61st row sees none."""
    if i % 61 == 60:
        return old + i + 1
    return old // 3 if i < 97 else old + (i // 97) * 97


def _visible(case, old, new):
    """(row, key) pairs that are visible, and the keys that some row sees."""
    pairs = 0
    L = old + new
    pre = min(case["prefix"], L)
    lo_all, seen_hi = L, 0
    for i in range(new):
        pos = old + i
        lo = max(0, pos - case["window"] + 1) if case["window"] else 0
        if case["docs"]:
            lo = max(lo, _doc(old, i))
        own_keys = max(0, pos + 1 - lo)
        pairs += own_keys + pre - max(0, min(pre, pos + 1) - lo)
        if own_keys:
            lo_all, seen_hi = min(lo_all, lo), max(seen_hi, pos + 1)
    return pairs, max(0, seen_hi - lo_all) + pre - max(0, min(pre, seen_hi) - lo_all)


def work(case):
    old, new = _lengths(case)
    P, hkv, g, d = case["page"], case["hkv"], case["g"], case["d"]
    if case["op"] == "evict":
        over = [a for a in old if a > case["above"]]
        kept = case["keep"] * len(over) * hkv
        # weights read, kept ones and kept codes in and out, and the read-back that shows them
        return {"bytes": 8 * len(old) + 4 * sum(over) * hkv + kept * (4 + 2 * (2 * d + 8 / P) + 2 * 3 * d), "flops": 0}
    seen = [_visible(case, a, b) for a, b in zip(old, new)]
    pairs, keys, rows = sum(p for p, _ in seen), sum(k for _, k in seen), sum(new) * hkv * g
    if case["op"] == "diff":
        return {"bytes": keys * hkv * (2 * d + 8 / P) + rows * (3 * d + 4), "flops": pairs * hkv * g * d * 4}
    touched = keys if case["decay"] == 1.0 and not case["whole"] else sum(a + b for a, b in zip(old, new))
    return {"bytes": keys * hkv * (d + 4 / P) + 8 * touched * hkv + rows * (2 * d + 4),
            "flops": pairs * hkv * g * d * 2}


# ---------------------------------------------------------------------------
# inputs

def _pools(phys, hkv, P, d, code, gen):
    """Codes and scales of K and of V; the rows of a page share a loudness that changes from page to page."""
    found = []
    for _ in range(2):
        x = torch.randn(phys, hkv, P, d, generator=gen, device="cuda")
        loud = torch.exp(0.3 * torch.randn(phys, hkv, generator=gen, device="cuda"))
        scale = x.abs().amax((2, 3)) / TOP[code]
        x = x / scale[:, :, None, None]
        x = torch.round(x).clamp(-127.0, 127.0).to(torch.int8) if code == "int8" else x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        found += [x, scale * loud]
    return found


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    old, new = _lengths(case)
    n, P, hkv, g, d, code = case["n"], case["page"], case["hkv"], case["g"], case["d"], case["code"]
    put = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = [a + b for a, b in zip(old, new)]
    used = [-(-a // P) for a in lens]
    per, phys, spare = max(used), sum(used), 7
    rows = torch.randperm(n + 1, generator=gen, device="cuda")[:n]  # which row of the table each sequence has
    u = torch.tensor(used, device="cuda")
    which = torch.repeat_interleave(rows, u, output_size=phys)
    at = torch.arange(phys, device="cuda") - torch.repeat_interleave(u.cumsum(0) - u, u, output_size=phys)
    perm = torch.randperm(phys + spare, generator=gen, device="cuda").int()
    table = torch.zeros(n + 1, per, dtype=torch.int32, device="cuda")
    table[which, at] = perm[spare:]
    long_lens = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    long_lens[rows] = put(lens)
    s = {"case": case, "rows": rows.int(), "table": table, "lens": long_lens, "handle": {}}
    s["k_pool"], s["k_scale"], s["v_pool"], s["v_scale"] = _pools(phys + spare, hkv, P, d, code, gen)
    if case["op"] != "diff":
        # weight that keys gathered before, spread over many factors of ten: about what these rows give
        s["weights"] = torch.exp(1.5 * torch.randn(phys + spare, hkv, P, generator=gen, device="cuda"))
        s["weights"] *= max(1, sum(new)) * g / sum(lens)
    if case["op"] == "evict":
        s["weights"][torch.rand(phys + spare, hkv, P, generator=gen, device="cuda") < case["zeros"]] = 0.0
        over = [b for b in range(n) if lens[b] > case["above"]]
        s |= {"over": put(over), "back_rows": s["rows"][put(over).long()], "back": put([case["keep"]] * len(over)),
              "back_start": put([case["keep"] * i for i in range(len(over))]), "back_first": put([0] * len(over)),
              "freed": sum(used[b] - -(-case["keep"] // P) for b in over), "free": perm.clone(), "free_count": put([spare]),
              "lens_out": long_lens.clone(), "count_out": put([0]), "weights_out": s["weights"].clone()}
        return s
    total, start = sum(new), [sum(new[:i]) for i in range(n)]
    # the queries are a slice of one projection's output
    qkv = torch.randn(total, (g + 2) * hkv, d, generator=gen, device="cuda").mul_(1.2).bfloat16()
    s |= {"total": total, "most": max(new), "start": put(start), "count": put(new), "q": qkv[:, :g * hkv]}
    if case["slopes"]:
        # geometric slopes; every other pair of heads has none
        h = torch.arange(hkv * g, device="cuda")
        s["slopes"] = torch.where(h % 4 < 2, torch.exp2(-8.0 * (h + 1) / (hkv * g)), torch.zeros(())).float()
    if case["prefix"]:
        s["prefix"] = put([min(case["prefix"], max(1, a)) for a in old])
    if case["docs"]:
        s["first_key"] = put([_doc(a, i) for a, b in zip(old, new) for i in range(b)])
    if case["op"] == "diff":
        # learned factors (a sigmoid's values) and a learned gain of the norm
        shape = (total, hkv * g // 2) if case["each"] else (hkv * g // 2,)
        s["lam"] = torch.sigmoid(torch.randn(shape, generator=gen, device="cuda"))
        s["gain"] = 0.2 * torch.exp(0.1 * torch.randn(d, generator=gen, device="cuda")) if case["norm"] else None
        return s
    # what the attention of these rows left behind: each row's log-sum-exp, or threshold
    s["tau"] = _rows_of(s, _statistic(_scores(s), case["alpha"]))
    s["coef"] = torch.rand(total, hkv * g, generator=gen, device="cuda") if case["coef"] else None
    s["fresh"] = put(lens) if case["whole"] else None
    return s


def _statistic(x, alpha):
    """[..., 1] of scores [..., T]: NaN where nothing is seen."""
    some = torch.isfinite(x).any(-1, keepdim=True)
    z = x * (alpha - 1.0) if alpha != 1.0 else x
    top = torch.where(some, z.amax(-1, keepdim=True), torch.zeros(()))
    if alpha == 1.0:
        tau = top + torch.log(torch.exp(z - top).sum(-1, keepdim=True))
    else:
        lo, hi = top - 1.0, top
        for _ in range(30):
            mid = (lo + hi) / 2
            more = (z - mid).clamp_min(0.0).pow(1.0 / (alpha - 1.0)).sum(-1, keepdim=True) >= 1.0
            lo, hi = torch.where(more, mid, lo), torch.where(more, hi, mid)
        tau = lo
    return torch.where(some, tau, torch.full((), math.nan, device="cuda"))


# ---------------------------------------------------------------------------
# the framework's calls

def _handle(s):
    """What a serving program keeps between its steps: the cache's view, output buffers, workspace."""
    h, c = s["handle"], s["case"]
    if h:
        return h
    from sparse_entmax_attention_gb300 import binding as B
    h["B"] = B
    h["cache"] = B.QuantCache.of(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"], s["lens"], c["g"])
    if c["op"] == "evict":
        h["pool"] = B.PagePool(s["free"], s["free_count"])
        h["ws"] = B.alloc_evict_workspace(h["cache"], c["n"], c["keep"])
        if len(s["over"]):
            h["back"] = B.Batch(s["back_start"], s["back"], len(s["over"]) * c["keep"], c["keep"], s["back_rows"])
            shape = (len(s["over"]) * c["keep"], c["hkv"], c["d"])
            h["k"], h["v"] = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return h
    h["batch"] = B.Batch(s["start"], s["count"], s["total"], s["most"], s["rows"])
    if c["op"] == "diff":
        h["out"] = B.alloc_diff_outputs(h["cache"], h["batch"])
        h["ws"] = B.alloc_attend_workspace(h["cache"], h["batch"])
    else:
        h["ws"] = B.alloc_weigh_workspace(h["cache"], h["batch"], c["alpha"])
    return h


def _own(s):
    h, c = _handle(s), s["case"]
    B = h["B"]
    if c["op"] == "evict":
        B.evict_q8(h["cache"], h["pool"], s["weights"], s["rows"], c["keep"], above=c["above"], sinks=c["sinks"],
                   recent=c["recent"], lens_out=s["lens_out"], count_out=s["count_out"], weights_out=s["weights_out"],
                   workspace=h["ws"])
        back = {}
        if len(s["over"]):
            B.read_q8(h["cache"], s["back_first"], h["back"], h["k"], h["v"])
            back = {"k": h["k"], "v": h["v"]}
        return {**back, "k_scale": s["k_scale"], "v_scale": s["v_scale"], "weights": s["weights_out"],
                "lens": s["lens_out"], "free": s["free"], "count": s["count_out"]}
    score = {"softcap": c["cap"], "slopes": s.get("slopes"), "window": c["window"], "prefix": s.get("prefix"),
             "first_key": s.get("first_key")}
    if c["op"] == "diff":
        o = B.attend_diff_q8(h["cache"], s["q"], s["lam"], h["batch"], gain=s["gain"], eps=EPS, workspace=h["ws"],
                             outputs=h["out"], **score)
        return {"out": o.out, "tau": o.tau}
    B.weigh_q8(h["cache"], s["weights"], s["q"], s["tau"], h["batch"], alpha=c["alpha"], coef=s["coef"], decay=c["decay"],
               fresh=s["fresh"], workspace=h["ws"], **score)
    return {"weights": s["weights"]}


# ---------------------------------------------------------------------------
# the plain forms

def _dense(pool, scale, table):
    """[n, hkv, tokens, d] of the pages in the table, as 32-bit values."""
    x = pool.view(torch.int8)[table].view(pool.dtype).float() * scale[table][..., None, None]
    n, per, hkv, P, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, per * P, d)


def _real(s):
    """[n, most]: the rows that are there, and where they lie."""
    i = torch.arange(s["most"], device="cuda")
    return i < s["count"].long()[:, None], (s["start"].long()[:, None] + i).clamp_max(s["total"] - 1)


def _scores(s):
    """[n, hkv, g, most, T], minus infinity where nothing is seen."""
    c = s["case"]
    hkv, g, d, most, n = c["hkv"], c["g"], c["d"], s["most"], c["n"]
    lens, table = s["lens"].long()[s["rows"].long()], s["table"].long()[s["rows"].long()]
    K = _dense(s["k_pool"], s["k_scale"], table)
    T = K.shape[2]
    real, row = _real(s)
    q = s["q"][row].float().view(n, most, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * most, d)
    x = (q @ K.transpose(2, 3)).view(n, hkv, g, most, T).mul_(1.0 / math.sqrt(d))
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    pos = (lens - s["count"].long())[:, None] + torch.arange(most, device="cuda")
    j = torch.arange(T, device="cuda")
    away = pos[:, :, None] - j
    if c["slopes"]:
        x = x - s["slopes"].view(1, hkv, g, 1, 1) * away.abs().float()[:, None, None]
    lo = torch.zeros_like(pos)
    if c["window"]:
        lo = torch.maximum(lo, pos - c["window"] + 1)
    if c["docs"]:
        lo = torch.maximum(lo, s["first_key"].long()[row])
    see = (away >= 0) & (j >= lo[:, :, None])
    if c["prefix"]:
        see = see | (j < torch.minimum(s["prefix"].long(), lens)[:, None, None])
    see = see & real[:, :, None]
    return x.masked_fill_(~see[:, None, None], -math.inf)


def _rows_of(s, x):
    """The rows that are there of [n, hkv, g, most, w], as [rows, heads] or [rows, heads, w]."""
    n, hkv, g, most, w = x.shape
    x = x.permute(0, 3, 1, 2, 4).reshape(n, most, hkv * g, w)[_real(s)[0]]
    return x[..., 0] if w == 1 else x


def _diff_plain(s):
    c = s["case"]
    hkv, g, d, most, n = c["hkv"], c["g"], c["d"], s["most"], c["n"]
    x = _scores(s)
    T = x.shape[-1]
    V = _dense(s["v_pool"], s["v_scale"], s["table"].long()[s["rows"].long()])
    some = torch.isfinite(x).any(-1, keepdim=True)
    top = torch.where(some, x.amax(-1, keepdim=True), torch.zeros(()))
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True, dtype=torch.float64)
    tau = torch.where(some, (top.double() + torch.log(total)).float(), torch.full((), math.nan, device="cuda"))
    p = p / torch.where(some, total.float(), torch.ones(()))
    o = _rows_of(s, (p.view(n, hkv, g * most, T) @ V).view(n, hkv, g, most, d))
    y = o[:, 0::2] - s["lam"][..., None] * o[:, 1::2]
    if c["norm"]:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * s["gain"]
    return {"out": y.bfloat16(), "tau": _rows_of(s, tau)}


def _weigh_plain(s):
    c = s["case"]
    hkv, g, most, n, P = c["hkv"], c["g"], s["most"], c["n"], c["page"]
    _, row = _real(s)
    spread = lambda v: v[row].view(n, most, hkv, g).permute(0, 2, 3, 1)[..., None]  # noqa: E731
    tau = spread(s["tau"])
    x = _scores(s)
    if c["alpha"] == 1.0:
        p = torch.exp(x - tau)
    else:
        p = (x * (c["alpha"] - 1.0) - tau).clamp_min(0.0).pow(1.0 / (c["alpha"] - 1.0))
    p = torch.where(torch.isfinite(tau) & torch.isfinite(x), p, torch.zeros(()))
    if s["coef"] is not None:
        p = p * spread(s["coef"])
    gives = p.sum((2, 3), dtype=torch.float64)                       # [n, hkv, T]
    lens, table = s["lens"].long()[s["rows"].long()], s["table"].long()[s["rows"].long()]
    j = torch.arange(x.shape[-1], device="cuda")
    before = s["weights"][table].permute(0, 2, 1, 3).reshape(n, hkv, -1)
    fresh = s["count"] if s["fresh"] is None else s["fresh"]
    held = (j < (lens - fresh.long())[:, None])[:, None] & (c["decay"] != 0.0)
    now = (torch.where(held, before.double() * c["decay"], 0.0) + gives).float()
    now = torch.where((j < lens[:, None])[:, None], now, before)
    used = torch.arange(table.shape[1], device="cuda") < ((lens + P - 1) // P)[:, None]
    s["weights"][table[used]] = now.view(n, hkv, -1, P).permute(0, 2, 1, 3)[used]
    return {"weights": s["weights"]}


def _e4m3(x):
    """The nearest e4m3 values (ties to the even one) of x, in 64 bits."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3.0)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _codes(q, code):
    """The code values nearest to q (64 bits)."""
    return torch.round(q).clamp(-127.0, 127.0) if code == "int8" else _e4m3(q)


def _move(s, pool, scale, table, src, over):
    """Keys src [m, hkv, keep] of the evicted sequences to the front of their pages; what lies there then."""
    c = s["case"]
    P, keep, hkv, d = c["page"], c["keep"], c["hkv"], c["d"]
    m, pages = len(over), -(-keep // P)
    src = torch.cat([src, src[..., -1:].expand(-1, -1, pages * P - keep)], -1)
    h = torch.arange(hkv, device="cuda")[None, :, None]
    page = table.gather(1, (src // P).view(m, -1)).view(m, hkv, -1)
    was = scale[page, h]
    real = (torch.arange(pages * P, device="cuda") < keep).view(pages, P)
    now = was.view(m, hkv, pages, P).amax(-1)                          # (the added ones are the last key again)
    by = (was.view(m, hkv, pages, P) / now[..., None]).double()
    x = pool.view(torch.int8)[page, h, src % P].view(pool.dtype).double().view(m, hkv, pages, P, d)
    x = _codes(x * by[..., None], c["code"])
    to = table[:, :pages]
    held = pool.view(torch.int8)[to].view(pool.dtype).double().permute(0, 2, 1, 3, 4)
    x = torch.where(real[..., None], x, held)
    stored = (x.to(torch.int8) if c["code"] == "int8" else x.float().to(torch.float8_e4m3fn)).view(torch.int8)
    pool.view(torch.int8)[to] = stored.permute(0, 2, 1, 3, 4)
    scale[to] = now.permute(0, 2, 1)
    value = (x.float() * now[..., None, None]).bfloat16().view(m, hkv, pages * P, d)[:, :, :keep]
    return value.permute(0, 2, 1, 3).reshape(m * keep, hkv, d)


def _evict_plain(s):
    c = s["case"]
    P, keep, hkv, over = c["page"], c["keep"], c["hkv"], s["over"].long()
    back = {}
    s["lens_out"].copy_(s["lens"])
    s["count_out"].copy_(s["free_count"] + s["freed"])
    if len(over):
        rows = s["rows"].long()[over]
        lens, table = s["lens"].long()[rows], s["table"].long()[rows]
        m, pages = len(over), -(-keep // P)
        w = s["weights"][table].permute(0, 2, 1, 3).reshape(m, hkv, -1)
        j = torch.arange(w.shape[-1], device="cuda")
        end = lens[:, None, None]
        rank = torch.where((j < c["sinks"]) | (j >= end - c["recent"]), torch.full((), math.inf, device="cuda"), w)
        rank = torch.where(j < end, rank, torch.full((), -math.inf, device="cuda"))
        src = rank.sort(dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values
        back = {"k": _move(s, s["k_pool"], s["k_scale"], table, src, over),
                "v": _move(s, s["v_pool"], s["v_scale"], table, src, over)}
        to = table[:, :pages]
        gone = s["weights_out"][to].permute(0, 2, 1, 3).reshape(m, hkv, -1)
        gone[..., :keep] = w.gather(-1, src)
        s["weights_out"][to] = gone.view(m, hkv, pages, P).permute(0, 2, 1, 3)
        s["lens_out"][rows] = keep
        # pages past the kept ones: sequences in order, each from its last page on
        have = (lens + P - 1) // P
        sums = (have - pages).cumsum(0)
        i = torch.arange(s["freed"], device="cuda")
        b = torch.searchsorted(sums, i, right=True)
        s["free"][s["free_count"].long() + i] = table[b, have[b] - 1 - (i - (sums - have + pages)[b])].int()
    return {**back, "k_scale": s["k_scale"], "v_scale": s["v_scale"], "weights": s["weights_out"], "lens": s["lens_out"],
            "free": s["free"], "count": s["count_out"]}


def run(state):
    if own:
        return _own(state)
    return {"diff": _diff_plain, "weigh": _weigh_plain, "evict": _evict_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions

def _nearest(q, code):
    """Codes nearest to q: whole numbers up to 127, or sign * 2^e * (8 + m)/8 with m in 0..7, e in -6..8."""
    a = q.abs()
    if code == "int8":
        low = torch.floor(a)
        more = a - low
        up = (more > 0.5) | ((more == 0.5) & (low % 2 == 1))
        v = torch.where(up, low + 1.0, low).clamp_max(127.0)
    else:
        grid = torch.tensor([k * 2.0 ** -9 for k in range(8)] +
                            [2.0 ** e * (8 + m) / 8 for e in range(-6, 9) for m in range(8)][:-1],
                            dtype=torch.float64, device=q.device)
        hi = torch.searchsorted(grid, a.contiguous()).clamp(1, len(grid) - 1)
        below, above = a - grid[hi - 1], grid[hi] - a
        v = torch.where((below < above) | ((below == above) & (hi % 2 == 1)), grid[hi - 1], grid[hi])
    return torch.where(q < 0, -v, v)


def _values(s, side, phys, h):
    """One KV head's [tokens, d] over the given pages."""
    pool, scale = s[side + "_pool"], s[side + "_scale"]
    x = pool.view(torch.int8)[phys, h].view(pool.dtype).double() * scale[phys, h].double()[:, None, None]
    return x.reshape(-1, pool.shape[-1])


def _exact_scores(s, b, old, new, start, h, K):
    """[new, L] of query head h and sequence b."""
    c = s["case"]
    pos = old + torch.arange(new, device="cuda")[:, None]
    j = torch.arange(old + new, device="cuda")[None]
    see = j <= pos
    if c["window"]:
        see &= pos - j < c["window"]
    if c["docs"]:
        see &= j >= s["first_key"][start:start + new, None]
    if c["prefix"]:
        see |= j < int(s["prefix"][b])
    x = s["q"][start:start + new, h].double() @ K.T / math.sqrt(c["d"])
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if c["slopes"]:
        x -= s["slopes"][h].double() * (pos - j).abs()
    return x.masked_fill_(~see, -math.inf), see.any(1)


def exact(case, seed):
    s = prepare(case, seed)
    old, new = _lengths(case)
    P, code, hkv, g, d = case["page"], case["code"], case["hkv"], case["g"], case["d"]
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    if case["op"] == "evict":
        keep, kept_pages = case["keep"], -(-case["keep"] // P)
        weights, scales = s["weights"].double(), {x: s[x + "_scale"].double() for x in "kv"}
        outs = {"k": [], "v": []}
        for b in s["over"].tolist():
            phys = s["table"][s["rows"][b]][:-(-old[b] // P)].long()
            values = {x: torch.zeros(keep, hkv, d, dtype=torch.float64, device="cuda") for x in "kv"}
            for h in range(hkv):
                w = s["weights"][phys, h].reshape(-1)[:old[b]].double()
                inner = w[case["sinks"]:old[b] - case["recent"]]
                take = keep - case["sinks"] - case["recent"]
                # those with fewer than `take` keys before them: heavier ones, or as heavy with a lower index
                kept = torch.zeros_like(inner, dtype=torch.bool)
                if take:
                    edge = torch.topk(inner, take).values[-1]
                    kept = inner > edge
                    level = (inner == edge).nonzero()[:, 0]
                    kept[level[:take - int(kept.sum())]] = True
                src = torch.cat([torch.arange(case["sinks"], device="cuda"), kept.nonzero()[:, 0] + case["sinks"],
                                 torch.arange(old[b] - case["recent"], old[b], device="cuda")])
                to = torch.arange(keep, device="cuda")
                weights[phys[to // P], h, to % P] = w[src]
                for x in "kv":
                    was = s[x + "_scale"][phys[src // P], h].double()
                    now = torch.zeros(kept_pages, dtype=torch.float64, device="cuda").scatter_reduce(0, to // P, was, "amax")
                    # the factor that a code is taken to a larger scale by is a 32-bit number
                    by = (was / now[to // P]).float().double()
                    pool = s[x + "_pool"]
                    held = pool.view(torch.int8)[phys[src // P], h, src % P].view(pool.dtype).double()
                    values[x][:, h] = _nearest(held * by[:, None], code) * now[to // P, None]
                    scales[x][phys[:kept_pages], h] = now
            for x in "kv":
                outs[x].append(values[x])
        back = {x: torch.cat(outs[x]) for x in "kv"} if outs["k"] else {}
        return {**back, "k_scale": scales["k"], "v_scale": scales["v"], "weights": weights, "lens": None, "free": None,
                "count": None}
    start, outs, taus = 0, [], []
    if case["op"] == "weigh":
        weights = s["weights"].double()
    for b in range(case["n"]):
        L, m = old[b] + new[b], new[b]
        phys = s["table"][s["rows"][b]][:-(-L // P)].long()
        at = torch.arange(L, device="cuda")
        o = torch.zeros(m, hkv * g, d, dtype=torch.float64, device="cuda")
        tau = torch.full((m, hkv * g), math.nan, dtype=torch.float64, device="cuda")
        for h in range(hkv):
            K = _values(s, "k", phys, h)[:L]
            V = _values(s, "v", phys, h)[:L] if case["op"] == "diff" else None
            gives = torch.zeros(L, dtype=torch.float64, device="cuda")
            for head in range(h * g, h * g + g):
                x, some = _exact_scores(s, b, old[b], m, start, head, K)
                if case["op"] == "diff":
                    tau[:, head] = torch.where(some, torch.logsumexp(x, 1), torch.full_like(zero, math.nan))
                    o[:, head] = torch.where(some[:, None], torch.exp(x - tau[:, head, None]), zero) @ V
                    continue
                t = s["tau"][start:start + m, head].double()[:, None]
                a1 = case["alpha"] - 1.0
                p = torch.exp(x - t) if a1 == 0.0 else (x * a1 - t).clamp_min(0.0).pow(1.0 / a1)
                p = torch.where(some[:, None], p, zero)
                gives += p.sum(0) if s["coef"] is None else s["coef"][start:start + m, head].double() @ p
            if case["op"] == "weigh":
                first = L - m if s["fresh"] is None else L - int(s["fresh"][b])
                before = weights[phys[at // P], h, at % P]
                weights[phys[at // P], h, at % P] = torch.where(at < first, before * case["decay"], zero) + gives
        outs.append(o)
        taus.append(tau)
        start += m
    if case["op"] == "weigh":
        return {"weights": weights}
    o = torch.cat(outs)
    y = o[:, 0::2] - s["lam"].double()[..., None] * o[:, 1::2]
    if case["norm"]:
        y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["gain"].double()
    return {"out": y, "tau": torch.cat(taus)}
