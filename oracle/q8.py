"""The 8-bit paged cache's operators in float64 on the CPU: page planning, the
quantising append, attention with its score forms and masks.

Oracle; test infrastructure only. The EntmaxKV pages describe no 8-bit cache;
these are the definitions of ``include/entmaxkv.h``, for one sequence or one
(sequence, KV head) at a time, with loops where the definition has them. Code
values (not bit patterns) are floats. Scales, and the factor that takes old
codes to a larger scale, are float32 numbers: they are stored or defined so.
"""

from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from . import entmax as em

TOP = {"int8": 127.0, "e4m3": 448.0}
FLOOR = 2.0 ** -96


def grid(code: str) -> np.ndarray:
    """The non-negative code values, ascending (index parity = last bit)."""
    if code == "int8":
        return np.arange(128, dtype=np.float64)
    sub = [k * 2.0 ** -9 for k in range(8)]
    nrm = [2.0 ** e * (8 + m) / 8 for e in range(-6, 9) for m in range(8)]
    return np.array(sub + nrm[:-1])  # the last pattern is NaN


def nearest(x, code: str) -> np.ndarray:
    """Code values nearest to x (float64), ties to the even pattern, saturating."""
    x = np.asarray(x, np.float64)
    g = grid(code)
    a = np.minimum(np.abs(x), g[-1])
    hi = np.clip(np.searchsorted(g, a), 1, len(g) - 1)
    below, above = a - g[hi - 1], g[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.copysign(np.where(up, g[hi], g[hi - 1]), x)


def nearest_exact(num: Fraction, code: str) -> float:
    """nearest() of an exact rational number."""
    a = min(abs(num), Fraction(float(grid(code)[-1])))
    g = [Fraction(float(v)) for v in grid(code)]
    best = min(range(len(g)), key=lambda i: (abs(g[i] - a), i % 2))
    return math.copysign(float(g[best]), num if num else 1)


def scale_of(amax, code: str) -> np.ndarray:
    return np.maximum(np.float32(np.asarray(amax, np.float64) / TOP[code]), np.float32(FLOOR)).astype(np.float64)


def append_page(codes, scale, n_old, new, code: str):
    """One (page, KV head, side): codes [P, d] held (the first n_old rows count), its scale, and the
    new rows [m, d] written behind them. Returns (codes, scale, any non-finite). The quotient is
    taken in float64: it lies within 2^-53 of the exact one, while a quotient that is no tie stays
    2^-33 or more away from every tie (24-bit scale, 8-bit value)."""
    codes, new = np.array(codes, np.float64), np.asarray(new, np.float64)
    fine = np.isfinite(new)
    amax = np.abs(np.where(fine, new, 0.0)).max() if new.size else 0.0
    s = float(scale_of(amax, code))
    if n_old and not s > scale:
        s = float(scale)
    elif n_old:
        r = float(np.float32(scale / s))
        codes[:n_old] = nearest(codes[:n_old] * r, code)
    x = np.where(np.isnan(new), 0.0, new)
    x = np.where(np.isinf(x), np.sign(x) * TOP[code] * s, x)
    codes[n_old:n_old + len(new)] = nearest(x / s, code)
    return codes, s, not fine.all()


def plan(lens, table, page, num_phys, free, seq_ids, n_new, total):
    """Pages, positions and slots of a batch, one slot after the other (host lists). Returns
    (table, lens, free, start, count, positions, slots, refused); inputs are not changed."""
    table, lens, free = [list(r) for r in table], list(lens), list(free)
    max_pages = len(table[0])
    start, count, positions, slots = [], [], [None] * total, [None] * total
    at, stopped, refused = 0, False, []
    for b, (seq, n) in enumerate(zip(seq_ids, n_new)):
        start.append(at)
        ok = n >= 0
        n = max(n, 0)
        if n == 0:
            count.append(0)
            if not ok:
                refused.append(b)
            continue
        ok = ok and 0 <= seq < len(lens) and lens[seq] + n <= max_pages * page
        if ok:
            L = lens[seq]
            need = -(-(L + n) // page) - -(-L // page)
            stopped = stopped or need > len(free)
            ok = not stopped and at + n <= total
        if ok:
            for j in range(need):
                table[seq][-(-L // page) + j] = free.pop()
            for i in range(n):
                pos = L + i
                positions[at + i] = pos
                slots[at + i] = table[seq][pos // page] * page + pos % page
            lens[seq] = L + n
        else:
            refused.append(b)
            for i in range(at, min(at + n, total)):
                positions[i] = slots[i] = -1
        count.append(n if ok else 0)
        at += n
    return table, lens, free, start, count, positions, slots, refused


def sees(L, count, window=0, prefix=0, first_key=None):
    """[count, L] which keys each of the last `count` tokens of L sees."""
    pos = np.arange(L - count, L)[:, None]
    j = np.arange(L)[None, :]
    lo = np.zeros((count, 1))
    if window > 0:
        lo = np.maximum(lo, pos - window + 1)
    if first_key is not None:
        lo = np.maximum(lo, np.asarray(first_key)[:, None])
    return ((j >= lo) & (j <= pos)) | (j < min(max(prefix, 0), L))


def attend(K, V, Q, alpha=1.0, scale=0.0, softcap=0.0, slope=0.0, window=0, prefix=0, first_key=None):
    """One query head of one sequence: K, V [L, d], Q [count, d] (its last tokens). Returns
    (out, tau, weights [count, L], scores)."""
    K, V, Q = (np.asarray(x, np.float64) for x in (K, V, Q))
    (L, d), count = K.shape, Q.shape[0]
    s = Q @ K.T * (scale if scale else 1.0 / math.sqrt(d))
    if softcap:
        s = softcap * np.tanh(s / softcap)
    s = s - slope * np.abs(np.arange(L - count, L)[:, None] - np.arange(L)[None, :])
    see = sees(L, count, window, prefix, first_key)
    P = np.zeros((count, L))
    tau = np.full(count, np.nan)
    for i in range(count):
        idx = np.nonzero(see[i])[0]
        if idx.size:
            P[i, idx], tau[i] = em.softmax(s[i, idx]) if alpha == 1.0 else em.entmax(s[i, idx], alpha)
    return P @ V, tau, P, np.where(see, s, -np.inf)


def difference(o0, o1, lam, gain=None, eps=0.0):
    """Of one pair's rows [count, d] and factors lam [count]: the difference, normalised over its head with a gain."""
    y = np.asarray(o0, np.float64) - np.asarray(lam, np.float64)[:, None] * np.asarray(o1, np.float64)
    if gain is None:
        return y
    return y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)


def key_weights(scores, tau, alpha=1.0):
    """[count, L] the weight that each row gives each key, from scores (minus infinity where a key is not seen) and the
    rows' statistics; rows whose statistic is not finite give nothing."""
    scores, tau = np.asarray(scores, np.float64), np.asarray(tau, np.float64)[:, None]
    fine = np.isfinite(tau) & np.isfinite(scores)
    x = np.where(fine, scores, 0.0) * (alpha - 1.0 if alpha != 1.0 else 1.0) - np.where(np.isfinite(tau), tau, 0.0)
    p = np.exp(np.where(fine, x, 0.0)) if alpha == 1.0 else np.maximum(x, 0.0) ** (1.0 / (alpha - 1.0))
    return np.where(fine, p, 0.0)


def kept_keys(w, keep, sinks=0, recent=0):
    """Of one KV head's weights [L]: the `keep` keys that stay, ascending."""
    L = len(w)
    if L <= keep:
        return list(range(L))
    rank = [math.inf if math.isnan(x) else float(x) for x in w]
    inner = sorted(range(sinks, L - recent), key=lambda j: (-rank[j], not math.isnan(w[j]), j))
    return sorted(list(range(sinks)) + inner[:keep - sinks - recent] + list(range(L - recent, L)))


def evict_rows(codes, scales, kept, page, code):
    """codes [L, d] of one (sequence, KV head, side), the scale of each key's page [L]: the kept keys' codes and the
    scales of the pages that they fill, in their order."""
    out, now = [], []
    for p0 in range(0, len(kept), page):
        src = kept[p0:p0 + page]
        s = max(float(scales[j]) for j in src)
        now.append(s)
        r = [1.0 if float(scales[j]) == s else float(np.float32(np.float32(scales[j]) / np.float32(s))) for j in src]
        out += [nearest(np.asarray(codes[j], np.float64) * x, code) for j, x in zip(src, r)]
    return np.array(out), now
