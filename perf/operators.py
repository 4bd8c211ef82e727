"""The operators of the 8-bit paged cache, case by case: page planning, the
quantising append with its read-back, and attention (softmax and alpha-entmax)
over the cache. `own` false computes each in elementary torch operations;
`own` true makes the calls a user makes of the framework.

Notation of the cases: `n` sequences, `hkv` KV heads of `g` query heads each,
head dimension `d`, pages of `page` tokens; cached lengths spread over
[len_lo, len_hi] and new tokens a sequence over [new_lo, new_hi], both the same
for every seed. A page and KV head has one float32 scale for K and one for V; a
stored value is code * scale.
"""

import math

import torch

own = False

FLOOR = 2.0 ** -96       # smallest scale
TOP = {"int8": 127.0, "e4m3": 448.0}


# ---------------------------------------------------------------------------
# cases

def _attn(name, code, n, len_lo, len_hi, new_lo, new_hi, hkv, g, d, page, alpha=1.0, cap=0.0, slopes=False,
          window=0, prefix=0, docs=False):
    c = {"op": "attend", "code": code, "n": n, "len_lo": len_lo, "len_hi": len_hi, "new_lo": new_lo,
         "new_hi": new_hi, "hkv": hkv, "g": g, "d": d, "page": page, "alpha": alpha, "cap": cap,
         "slopes": slopes, "window": window, "prefix": prefix, "docs": docs}
    return {"name": name, **c} if name else c


def _write(name, code, n, len_lo, len_hi, new_lo, new_hi, hkv, g, d, page):
    c = {"op": "write", "code": code, "n": n, "len_lo": len_lo, "len_hi": len_hi, "new_lo": new_lo,
         "new_hi": new_hi, "hkv": hkv, "g": g, "d": d, "page": page}
    return {"name": name, **c} if name else c


def _plan(name, n, len_lo, len_hi, new_lo, new_hi, page, short=False):
    c = {"op": "plan", "n": n, "len_lo": len_lo, "len_hi": len_hi, "new_lo": new_lo, "new_hi": new_hi,
         "page": page, "short": short}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a decode step of a running batch: most sequences need no page, a few one
        _plan("plan a decode step", 64, 100, 30000, 1, 1, 32),
        # admission of a queue of prompts into a pool that cannot hold them all
        _plan("plan a queue of prompts", 333, 1, 4000, 0, 700, 16, short=True),
        # the tokens of one decode step, each into a partly filled page
        _write("write a decode step", "int8", 64, 100, 30000, 1, 1, 8, 4, 128, 32),
        # the chunks of a continuous batch: decodes and prompt pieces together
        _write("write a mixed batch", "e4m3", 37, 1, 9000, 1, 1000, 8, 4, 64, 16),
        # one long prompt behind a page that is not full
        _write("write a prompt", "int8", 1, 77, 77, 32801, 32801, 8, 4, 128, 32),
        # one user's next token: latency
        _attn("decode one sequence", "int8", 1, 32768, 32768, 1, 1, 8, 4, 128, 32),
        # batched serving, lengths far apart, capped scores, linear distance bias
        _attn("decode a ragged batch", "e4m3", 16, 4096, 65536, 1, 1, 8, 4, 128, 16, cap=30.0, slopes=True),
        # several drafted tokens checked at once, sliding window with a kept prefix
        _attn("check drafted tokens", "int8", 24, 1000, 20000, 2, 5, 4, 8, 64, 32, window=4096, prefix=100),
        # a prompt's chunk against a long context
        _attn("a chunk of a long prompt", "int8", 1, 30001, 30001, 2048, 2048, 8, 4, 128, 32, cap=50.0),
        # ragged chunks, several documents in a sequence, a prefix that all see, distance bias
        _attn("ragged chunks", "e4m3", 6, 500, 8000, 60, 1500, 8, 4, 128, 16, slopes=True, prefix=200, docs=True),
        # entmax decode of a long context with a distance bias on the heads
        _attn("entmax decode of a long context", "int8", 1, 131072, 131072, 1, 1, 8, 4, 128, 32, alpha=1.5, slopes=True),
        # entmax decode of a batch
        _attn("entmax decode of a batch", "e4m3", 16, 1000, 32000, 1, 1, 8, 4, 128, 16, alpha=2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "write", "decode", "decode", "chunk", "entmax"])
    code, page, d = rng.choice(["int8", "e4m3"]), rng.choice([16, 32]), rng.choice([64, 128])
    hkv, g = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if kind == "plan":
        n = _log(rng, 1, 1000)
        new = _log(rng, 1, 1000)
        lo = _log(rng, 1, 2000)
        return _plan(None, n, lo, lo + _log(rng, 1, 20000), rng.choice([0, 1, new]), new, page, rng.random() < 0.3)
    if kind == "write":
        n = _log(rng, 1, 64)
        new = _log(rng, 1, 32000 // n)
        lo = _log(rng, 1, 3000)
        return _write(None, code, n, lo, lo + _log(rng, 1, 6000), rng.choice([1, new]), new, hkv, g, d, page)
    cap = rng.choice([0.0, 0.0, rng.uniform(5.0, 60.0)])
    slopes, docs = rng.random() < 0.4, rng.random() < 0.25
    window = rng.choice([0, 0, _log(rng, 1, 5000)])
    prefix = rng.choice([0, 0, _log(rng, 1, 400)])
    if kind == "chunk":
        n = _log(rng, 1, 8)
        new = _log(rng, 6, 2000 // n)
        lo = _log(rng, 1, 4000)
        return _attn(None, code, n, lo, lo + _log(rng, 1, 16000), rng.choice([1, new]), new, hkv, min(g, 4), d, page,
                     1.0, cap, slopes, window, prefix, docs)
    n = _log(rng, 1, 64)
    hi = _log(rng, 2, min(131072, 360000 // n))
    lo = max(1, hi // rng.choice([1, 3, 10, 100]))
    if kind == "entmax":
        return _attn(None, code, n, lo, hi, 1, 1, hkv, g, d, page, rng.choice([1.5, 2.0]), cap, slopes, window,
                     prefix, docs)
    new = rng.choice([1, 1, 1, 2, 4, 8])
    return _attn(None, code, n, lo, hi, 1, new, hkv, g, d, page, 1.0, cap, slopes, window, prefix, docs)


def _spread(n, lo, hi, turn):
    """n whole numbers over [lo, hi], far apart ones next to each other."""
    if n == 1:
        return [hi]
    a = math.log(lo + 1.0)
    b = math.log(hi + 1.0)
    v = [min(hi, max(lo, int(round(math.exp(a + (b - a) * i / (n - 1)) - 1.0)) - (i * 7) % 3)) for i in range(n)]
    step = next(s for s in range(turn, turn + n + 2) if math.gcd(s, n) == 1)
    return [v[(i * step) % n] for i in range(n)]


def _lengths(case):
    """(cached tokens before, new tokens) of each sequence."""
    return (_spread(case["n"], case["len_lo"], case["len_hi"], 5),
            _spread(case["n"], case["new_lo"], case["new_hi"], 3))


def _visible(case, old, new):
    """Of each sequence: the (row, key) pairs that are visible, and the keys that some row sees."""
    pairs = keys = 0
    L = old + new
    pre = min(case["prefix"], L)
    lo_all, seen_hi = L, 0
    for i in range(new):
        pos = old + i
        lo = 0
        if case["window"]:
            lo = max(lo, pos - case["window"] + 1)
        if case["docs"]:
            lo = max(lo, _doc(old, i))
        own_keys = max(0, pos + 1 - lo)
        both = max(0, min(pre, pos + 1) - lo)
        pairs += own_keys + pre - both
        if own_keys:
            lo_all, seen_hi = min(lo_all, lo), max(seen_hi, pos + 1)
    keys = max(0, seen_hi - lo_all) + pre - max(0, min(pre, seen_hi) - lo_all)
    return pairs, keys


def _doc(old, i):
    """First key of the document that new token i belongs to: every 97 new tokens another one begins."""
    return old // 3 if i < 97 else old + (i // 97) * 97


def work(case):
    old, new = _lengths(case)
    n, P = case["n"], case["page"]
    tokens = sum(new)
    if case["op"] == "plan":
        pages = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(old, new))
        return {"bytes": 24 * n + 8 * pages + 12 * tokens, "flops": 0}
    hkv, g, d = case["hkv"], case["g"], case["d"]
    if case["op"] == "write":
        touched = sum(-(-(a + b) // P) - a // P for a, b in zip(old, new))
        back = sum(a + b - a // P * P for a, b in zip(old, new))
        held = back - tokens  # tokens that a partly filled page held before
        return {"bytes": 2 * hkv * (d * (2 * tokens + tokens + held + 3 * back) + 8 * touched), "flops": 0}
    seen = [_visible(case, a, b) for a, b in zip(old, new)]
    rows = tokens * hkv * g
    # entmax reads K whole; of V only what gets weight, which is not counted
    sides = 1 if case["alpha"] > 1.0 else 2
    return {"bytes": sum(k for _, k in seen) * hkv * (d + 4 / P) * sides + rows * (4 * d + 4),
            "flops": sum(p for p, _ in seen) * hkv * g * d * 2 * sides}


# ---------------------------------------------------------------------------
# inputs

def _e4m3(x):
    """The nearest e4m3 values (ties to the even one) of x, in 64 bits."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3.0)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _codes(q, code):
    """The code values nearest to q (64 bits)."""
    return torch.round(q).clamp(-127.0, 127.0) if code == "int8" else _e4m3(q)


def _scale_of(amax, code):
    return (amax.double() / TOP[code]).float().clamp_min(FLOOR)


def _stored(values, code):
    return values.to(torch.int8) if code == "int8" else values.float().to(torch.float8_e4m3fn)


def _pages_of(case):
    old, new = _lengths(case)
    return max(-(-(a + b) // case["page"]) for a, b in zip(old, new))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    old, new = _lengths(case)
    n, P = case["n"], case["page"]
    put = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    total = sum(new)
    per = _pages_of(case)
    start = [sum(new[:i]) for i in range(n)]
    s = {"case": case, "total": total, "most": max(new), "handle": {}}
    if case["op"] == "plan":
        need = [-(-(a + b) // P) - -(-a // P) for a, b in zip(old, new)]
        have = [-(-a // P) for a in old]
        pool = sum(have) + sum(need) + 5
        perm = torch.randperm(pool, generator=gen, device="cuda").int()
        free = sum(need) * 2 // 3 if case["short"] else sum(need) + 5
        table = torch.full((n + 2, per + 1), -1, dtype=torch.int32, device="cuda")
        rows = torch.randperm(n + 2, generator=gen, device="cuda")[:n]  # which row of the table each sequence has
        h = torch.tensor(have, device="cuda")
        flat = torch.repeat_interleave(rows * (per + 1), h, output_size=sum(have))
        at = torch.arange(sum(have), device="cuda") - torch.repeat_interleave(h.cumsum(0) - h, h, output_size=sum(have))
        table.view(-1)[flat + at] = perm[pool - sum(have):]
        lens = torch.zeros(n + 2, dtype=torch.int32, device="cuda")
        lens[rows] = put(old)
        return {**s, "table": table, "lens": lens, "rows": rows.int(), "new": put(new), "pool": pool,
                "free": perm[:pool].contiguous(), "free_count": put([free]),
                "lens_out": lens.clone(), "count_out": put([0])}
    hkv, g, d, code = case["hkv"], case["g"], case["d"], case["code"]
    used = [-(-(a + b) // P) for a, b in zip(old, new)]
    phys = sum(used)
    table = torch.zeros(n, per, dtype=torch.int32, device="cuda")
    u = torch.tensor(used, device="cuda")
    row = torch.repeat_interleave(torch.arange(n, device="cuda"), u, output_size=phys)
    at = torch.arange(phys, device="cuda") - torch.repeat_interleave(u.cumsum(0) - u, u, output_size=phys)
    table[row, at] = torch.randperm(phys, generator=gen, device="cuda").int()
    # keys and values of a page share a loudness that changes from page to page
    pools = []
    for _ in range(2):
        x = torch.randn(phys, hkv, P, d, generator=gen, device="cuda")
        loud = torch.exp(0.3 * torch.randn(phys, hkv, generator=gen, device="cuda"))
        scale = _scale_of(x.abs().amax((2, 3)), code)
        if code == "int8":
            x = torch.round(x / scale[:, :, None, None]).clamp(-127.0, 127.0)
        else:
            x = (x / scale[:, :, None, None]).clamp(-448.0, 448.0)
        pools += [x.to(torch.int8 if code == "int8" else torch.float8_e4m3fn), scale * loud]
        del x
    # q, k and v of the new tokens are slices of one projection's output
    qkv = torch.randn(total, (g + 2) * hkv, d, generator=gen, device="cuda").mul_(1.2).bfloat16()
    s |= {"k_pool": pools[0], "k_scale": pools[1], "v_pool": pools[2], "v_scale": pools[3], "table": table,
          "lens": put([a + b for a, b in zip(old, new)]), "start": put(start), "count": put(new),
          "q": qkv[:, :g * hkv], "k": qkv[:, g * hkv:g * hkv + hkv], "v": qkv[:, g * hkv + hkv:]}
    if case["op"] == "write":
        first = [a // P * P for a in old]
        back = [a + b - f for a, b, f in zip(old, new, first)]
        s |= {"old": put(old), "first": put(first), "back": put(back), "back_total": sum(back), "back_most": max(back),
              "back_start": put([sum(back[:i]) for i in range(n)]),
              "touched": sum(-(-(a + b) // P) - a // P for a, b in zip(old, new))}
        return s
    if case["slopes"]:
        # geometric slopes; every other head has none
        h = torch.arange(hkv * g, device="cuda")
        s["slopes"] = torch.where(h % 2 == 0, torch.exp2(-8.0 * (h + 1) / (hkv * g)), torch.zeros(())).float()
    if case["prefix"]:
        s["prefix"] = put([min(case["prefix"], max(1, a)) for a in old])
    if case["docs"]:
        s["first_key"] = put([_doc(a, i) for a, b in zip(old, new) for i in range(b)])
    return s


# ---------------------------------------------------------------------------
# the framework's calls

def _handle(s):
    """What a serving program keeps between its steps: the cache's view, output buffers, workspace."""
    h, c = s["handle"], s["case"]
    if h:
        return h
    from sparse_entmax_attention_gb300 import binding as B
    h["B"] = B
    if c["op"] == "plan":
        h["pages"] = B.PageTable(s["table"], s["lens"], c["page"], s["pool"])
        h["pool"] = B.PagePool(s["free"], s["free_count"])
        h["plan"] = B.alloc_plan(c["n"], s["total"], "cuda")
        return h
    h["cache"] = B.QuantCache.of(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"], s["lens"], c["g"])
    h["batch"] = B.Batch(s["start"], s["count"], s["total"], s["most"])
    if c["op"] == "write":
        h["back"] = B.Batch(s["back_start"], s["back"], s["back_total"], s["back_most"])
        shape = (s["back_total"], c["hkv"], c["d"])
        h["k"], h["v"] = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return h
    h["out"] = B.alloc_attend_outputs(h["cache"], h["batch"])
    h["ws"] = B.alloc_attend_workspace(h["cache"], h["batch"], c["alpha"])
    return h


def _own(s):
    h, c = _handle(s), s["case"]
    B = h["B"]
    if c["op"] == "plan":
        p = B.plan_pages(h["pages"], h["pool"], s["new"], h["plan"], seq_ids=s["rows"], lens_out=s["lens_out"],
                         count_out=s["count_out"])
        return {"start": p.start, "count": p.count, "positions": p.positions, "slots": p.slots, "table": s["table"],
                "lens": s["lens_out"], "free": s["count_out"]}
    if c["op"] == "write":
        B.append_q8(h["cache"], s["k"], s["v"], h["batch"])
        B.read_q8(h["cache"], s["first"], h["back"], h["k"], h["v"])
        return {"k": h["k"], "v": h["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    o = B.attend_q8(h["cache"], s["q"], h["batch"], alpha=c["alpha"], softcap=c["cap"], slopes=s.get("slopes"),
                    window=c["window"], prefix=s.get("prefix"), first_key=s.get("first_key"), workspace=h["ws"],
                    outputs=h["out"])
    return {"out": o.out, "tau": o.tau}


# ---------------------------------------------------------------------------
# the plain forms

def _plan_plain(s):
    c, P = s["case"], s["case"]["page"]
    rows, new = s["rows"].long(), s["new"].long()
    L = s["lens"][rows].long()
    have = (L + P - 1) // P
    need = (L + new + P - 1) // P - have
    sums = need.cumsum(0)
    ok = sums <= s["free_count"].long()
    take = torch.where(ok, need, torch.zeros_like(need))
    begin = sums - need
    start = new.cumsum(0) - new
    count = torch.where(ok, new, torch.zeros_like(new))
    # pages: entry j of the plan goes to the slot whose range holds it
    j = torch.arange(s["pool"], device="cuda")
    slot = torch.searchsorted(sums, j, right=True).clamp_max(c["n"] - 1)
    used = (j < take.sum()) & (j >= begin[slot])
    table, width = s["table"], s["table"].shape[1]
    at = rows[slot] * width + have[slot] + (j - begin[slot])
    page = s["free"][(s["free_count"].long() - 1 - j).clamp_min(0)]
    flat = torch.cat([table.view(-1), table.new_zeros(1)])
    flat[torch.where(used, at, torch.full_like(at, table.numel()))] = page
    table.copy_(flat[:-1].view_as(table))
    # tokens
    t = torch.arange(s["total"], device="cuda")
    slot = torch.searchsorted(start + new, t, right=True).clamp_max(c["n"] - 1)
    pos = L[slot] + t - start[slot]
    phys = table[rows[slot], (pos // P).clamp_max(width - 1)].long()
    fine = ok[slot]
    s["lens_out"].copy_(s["lens"])
    s["lens_out"][rows] = (L + count).int()
    s["count_out"].copy_((s["free_count"].long() - take.sum()).int())
    minus = torch.full_like(pos, -1)
    return {"start": start.int(), "count": count.int(), "positions": torch.where(fine, pos, minus).int(),
            "slots": torch.where(fine, phys * P + pos % P, minus), "table": table, "lens": s["lens_out"],
            "free": s["count_out"]}


def _write_plain(s):
    c, P, code = s["case"], s["case"]["page"], s["case"]["code"]
    old, lens, start = s["old"].long(), s["lens"].long(), s["start"].long()
    first = old // P
    pages = (lens + P - 1) // P - first
    slot = torch.repeat_interleave(torch.arange(c["n"], device="cuda"), pages, output_size=s["touched"])
    lp = first[slot] + torch.arange(s["touched"], device="cuda") - (pages.cumsum(0) - pages)[slot]
    phys = s["table"][slot, lp].long()
    pos = lp[:, None] * P + torch.arange(P, device="cuda")
    is_new = (pos >= old[slot, None]) & (pos < lens[slot, None])
    is_old = pos < old[slot, None]
    src = (start[slot, None] + pos - old[slot, None]).clamp(0, s["total"] - 1)
    back = {}
    for x, pool, scale, name in ((s["k"], s["k_pool"], s["k_scale"], "k"), (s["v"], s["v_pool"], s["v_scale"], "v")):
        rows = x[src].float().permute(0, 2, 1, 3)                       # [pages, hkv, P, d]
        fresh, held = is_new[:, None, :, None], is_old[:, None, :, None]
        amax = torch.where(fresh, rows.abs(), torch.zeros(())).amax((2, 3))
        before = torch.where(is_old.any(1)[:, None], scale[phys], torch.zeros(()))
        now = torch.maximum(_scale_of(amax, code), before)
        ratio = before / now
        was = pool.view(torch.int8)[phys].view(pool.dtype)
        again = _codes(was.double() * ratio.double()[:, :, None, None], code)
        codes = _codes(rows.double() / now.double()[:, :, None, None], code)
        stored = torch.where(fresh, codes, torch.where(held, again, was.double()))
        pool.view(torch.int8)[phys] = _stored(stored, code).view(torch.int8)
        scale[phys] = now
        values = (stored.float() * now[:, :, None, None]).bfloat16()
        keep = is_new | is_old
        back[name] = values.permute(0, 2, 1, 3)[keep]
    return {"k": back["k"], "v": back["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _dense(pool, scale, table):
    """[n, hkv, tokens, d] of the pages in the table, as 32-bit values."""
    x = pool.view(torch.int8)[table.long()].view(pool.dtype).float() * scale[table.long()][..., None, None]
    n, per, hkv, P, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, per * P, d)


def _attend_plain(s):
    c = s["case"]
    hkv, g, d, most = c["hkv"], c["g"], c["d"], s["most"]
    n, Hq = c["n"], hkv * g
    lens, start, count = s["lens"].long(), s["start"].long(), s["count"].long()
    K = _dense(s["k_pool"], s["k_scale"], s["table"])
    V = _dense(s["v_pool"], s["v_scale"], s["table"])
    T = K.shape[2]
    i = torch.arange(most, device="cuda")
    row = (start[:, None] + i).clamp_max(s["total"] - 1)               # [n, most]
    real = i < count[:, None]
    q = s["q"][row].float().view(n, most, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * most, d)
    x = (q @ K.transpose(2, 3)).view(n, hkv, g, most, T)
    x = x * (1.0 / math.sqrt(d))
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    pos = (lens - count)[:, None] + i                                   # [n, most]
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
    x = torch.where(see[:, None, None], x, torch.full((), -math.inf, device="cuda"))
    some = see.any(-1)[:, None, None, :, None]
    if c["alpha"] == 1.0:
        top = torch.where(some, x.amax(-1, keepdim=True), torch.zeros(()))
        p = torch.exp(x - top)
        total = p.double().sum(-1, keepdim=True)
        tau = (top.double() + torch.log(total)).float()
        p = p / torch.where(some, total.float(), torch.ones(()))
    else:
        z = x * (c["alpha"] - 1.0)
        top = torch.where(some, z.amax(-1, keepdim=True), torch.zeros(()))
        y, _ = (z - top).clamp_min(-1.0).double().sort(-1, descending=True)   # nothing at or below -1 has weight
        k = torch.arange(1, T + 1, device="cuda")
        m = y.cumsum(-1) / k
        if c["alpha"] == 2.0:
            t = m - 1.0 / k
        else:
            var = (y.square().cumsum(-1) / k - m.square()) * k
            t = m - ((1.0 - var) / k).clamp_min(0.0).sqrt()
        kept = ((t <= y) & (y > -1.0)).sum(-1, keepdim=True).clamp_min(1)
        t = t.gather(-1, kept - 1)
        p = ((z - top).double() - t).clamp_min(0.0)
        p = (p if c["alpha"] == 2.0 else p.square()).float()
        tau = (top.double() + t).float()
    tau = torch.where(some, tau, torch.full((), math.nan, device="cuda"))[..., 0]
    o = (p.reshape(n, hkv, g * most, T) @ V).view(n, hkv, g, most, d)
    o = torch.where(some, o, torch.zeros(()))
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(n, most, Hq, d)[real].bfloat16(),
            "tau": tau.permute(0, 3, 1, 2).reshape(n, most, Hq)[real]}


def run(state):
    if own:
        return _own(state)
    return {"plan": _plan_plain, "write": _write_plain, "attend": _attend_plain}[state["case"]["op"]](state)


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


def _whole(pool, scale, phys, h):
    """One KV head's [tokens, d] over the given pages."""
    x = pool.view(torch.int8)[phys, h].view(pool.dtype).double() * scale[phys, h].double()[:, None, None]
    return x.reshape(-1, pool.shape[-1])


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    old, new = _lengths(case)
    P, code, hkv, g, d = case["page"], case["code"], case["hkv"], case["g"], case["d"]
    start = 0
    outs = []
    if case["op"] == "write":
        table = s["table"].cpu()
        scales = [s["k_scale"].double(), s["v_scale"].double()]
        for b in range(case["n"]):
            lp = torch.arange(old[b] // P, -(-(old[b] + new[b]) // P))
            phys = table[b, lp].long().cuda()
            keep = old[b] % P
            pair = []
            for side, (x, pool, scale) in enumerate(((s["k"], s["k_pool"], s["k_scale"]),
                                                     (s["v"], s["v_pool"], s["v_scale"]))):
                page = torch.zeros(len(lp) * P, hkv, d, dtype=torch.float64, device="cuda")
                page[keep:keep + new[b]] = x[start:start + new[b]].double()
                page = page.view(len(lp), P, hkv, d)
                # stored scales, and the factor that old codes are taken to a larger scale by, are 32-bit numbers
                sc = torch.clamp((page.abs().amax((1, 3)) / TOP[code]).float().double(), min=FLOOR)
                if keep:
                    sc[0] = torch.maximum(sc[0], scale[phys[0]].double())
                val = _nearest(page / sc[:, None, :, None], code)
                if keep:
                    by = (scale[phys[0]].double() / sc[0]).float().double()
                    val[0, :keep] = _nearest(pool[phys[0].item(), :, :keep].double() * by[:, None, None], code).transpose(0, 1)
                scales[side][phys] = sc
                pair.append((val * sc[:, None, :, None]).view(-1, hkv, d)[:keep + new[b]])
            outs.append(pair)
            start += new[b]
        return {"k": torch.cat([o[0] for o in outs]), "v": torch.cat([o[1] for o in outs]),
                "k_scale": scales[0], "v_scale": scales[1]}
    taus = []
    for b in range(case["n"]):
        L, m = old[b] + new[b], new[b]
        phys = s["table"][b, :-(-L // P)].long()
        o = torch.zeros(m, hkv * g, d, dtype=torch.float64, device="cuda")
        tau = torch.full((m, hkv * g), math.nan, dtype=torch.float64, device="cuda")
        pos = old[b] + torch.arange(m, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        see = j <= pos
        if case["window"]:
            see &= pos - j < case["window"]
        if case["docs"]:
            see &= j >= s["first_key"][start:start + m, None]
        if case["prefix"]:
            see |= j < int(s["prefix"][b])
        for h in range(hkv * g):
            k, v = (_whole(s[p + "_pool"], s[p + "_scale"], phys, h // g)[:L] for p in "kv")
            x = s["q"][start:start + m, h].double() @ k.T / math.sqrt(d)
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case["slopes"]:
                x -= s["slopes"][h].double() * (pos - j).abs()
            x.masked_fill_(~see, -math.inf)
            some = see.any(1)
            if case["alpha"] == 1.0:
                tau[:, h] = torch.logsumexp(x, 1)
                p = torch.exp(x - tau[:, h, None])
            else:  # the threshold by bisection: the weights' sum falls from at least 1 to 0 over [max - 1, max]
                z, power = x * (case["alpha"] - 1.0), 1.0 / (case["alpha"] - 1.0)
                hi = z.amax(1, keepdim=True)
                lo = hi - 1.0
                for _ in range(60):
                    mid = (lo + hi) / 2
                    more = (z - mid).clamp_min(0.0).pow(power).sum(1, keepdim=True) >= 1.0
                    lo, hi = torch.where(more, mid, lo), torch.where(more, hi, mid)
                tau[:, h] = lo[:, 0]
                p = (z - lo).clamp_min(0.0).pow(power)
            p = torch.where(some[:, None], p, torch.zeros((), dtype=torch.float64, device="cuda"))
            tau[:, h] = torch.where(some, tau[:, h], torch.full((), math.nan, dtype=torch.float64, device="cuda"))
            o[:, h] = p @ v
        outs.append(o)
        taus.append(tau)
        start += m
    return {"out": torch.cat(outs), "tau": torch.cat(taus)}
