"""Shared by the 8-bit cache's GPU tests: caches with given lengths over
shuffled pages, and the oracle's answer for a whole batch."""

from __future__ import annotations

import numpy as np
import torch

from oracle import q8 as oq
from sparse_entmax_attention_gb300 import binding as B

DT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def empty_cache(code, lens, hkv=2, g=4, d=128, P=32, spare=3, seed=0, garbage=False):
    """A QuantCache with shuffled pages for the given lengths. garbage: codes and scales start as
    bytes that stand for NaN (e4m3) or the type's lowest value (int8), scales as NaN."""
    per = max(-(-n // P) for n in lens) + 1
    pages = sum(-(-n // P) for n in lens) + spare
    c = B.QuantCache(hkv, g, d, P, len(lens), per, pages, DT[code])
    if garbage:
        for pool in (c.k_pool, c.v_pool):
            pool.view(torch.uint8).fill_(0xff if code == "e4m3" else 0x80)
        c.k_scale.fill_(float("nan"))
        c.v_scale.fill_(float("nan"))
    perm = np.random.default_rng(seed).permutation(pages)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // P)
        c.block_table[b, :m] = i32(perm[at:at + m].tolist())
        at += m
    c.seq_lens.copy_(i32(lens))
    return c


def batch_of(counts, seq_ids=None, gap=0):
    """A Batch of consecutive slots, `gap` unowned rows behind each."""
    start = [sum(counts[:b]) + gap * b for b in range(len(counts))]
    return B.Batch(i32(start), i32(counts), sum(counts) + gap * len(counts), max(counts + [1]),
                   None if seq_ids is None else i32(seq_ids))


def values(pool, scale):
    return pool.float().double() * scale.double()[..., None, None]


def dense(c, b, h, side):
    """[L, d] float64 of one sequence and KV head."""
    pool, scale = (c.k_pool, c.k_scale) if side == "k" else (c.v_pool, c.v_scale)
    P, L = c.cfg.page_size, int(c.seq_lens[b])
    ph = c.block_table[b, :-(-L // P)].long()
    x = pool.view(torch.int8)[ph, h].view(pool.dtype).float().double() * scale[ph, h].double()[:, None, None]
    return x.reshape(-1, c.cfg.head_dim)[:L].cpu().numpy()


def v_scales(c, b, h):
    """[L] float64: the V scale of each token's page."""
    P, L = c.cfg.page_size, int(c.seq_lens[b])
    ph = c.block_table[b, :-(-L // P)].long()
    return np.repeat(c.v_scale[ph, h].double().cpu().numpy(), P)[:L]


def filled(code, lens, counts, seed=0, loud=1.0, **kw):
    """A cache whose sequences hold random tokens (through append_q8)."""
    c = empty_cache(code, lens, seed=seed, **kw)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    total = sum(lens)
    hkv, d = c.cfg.num_kv_heads, c.cfg.head_dim
    if total:
        k = torch.randn(total, hkv, d, generator=gen, device="cuda").mul_(loud).bfloat16()
        v = torch.randn(total, hkv, d, generator=gen, device="cuda").bfloat16()
        B.append_q8(c, k, v, batch_of(list(lens)))
    q = torch.randn(sum(counts), c.num_q_heads, d, generator=gen, device="cuda").bfloat16()
    return c, q


def check_attend(c, q, counts, o, seq_ids=None, alpha=1.0, start=None, scale=0.0, softcap=0.0,
                 slopes=None, window=0, prefix=None, first_key=None):
    """Compare rows with the oracle. Bounds, per element of a row's output o = Σ p v:
      2^-8·|o|           the rounding to bf16 (half a step),
      2^-11·Σ p|v|       each weight's rounding to a half before it meets V (half a step),
      and what a half keeps of a small one: a weight times its page's V scale s meets the codes c (v = s·c) as a
      half, whose spacing below 2^-14 is 2^-24, so rounding moves it by up to 2^-25.
        softmax: the row's largest p·s lies at 2^8 or above (2^{t − M + 8} with M at most the largest t), so that
                 is at most 2^-33·max(p·s) for each key seen: 2^-33·max(p·s)·Σ|c|;
        entmax:  of 32 keys the largest p is brought to 1/2 or above, and its s/max(s) is at most 1: at most
                 2^-24·max(p)·max(s) for each key of the support: 2^-24·max(p)·max(s)·Σ|c| over the support,
      δ-terms            a score off by δ = 2^-20·(Σ|q||k|·scale + slope·L + cap) + 2^-20 (fp32 sums of d
                         products, a few further fp32 operations and 2^-22 functions) moves a softmax
                         weight by 2δp; an entmax weight [z−τ]^β by at most β·(y+δz)^{β−1}·δz for β ≥ 1
                         and δz^β below, δz = 2(α−1)δ (τ moves no further than the scores), counted over
                         every key within δz of the support.
    τ is held to 2δ (softmax: log-sum-exp moves no further than its scores; its own fp32 rounding is
    2^-23·|τ|)."""
    G, d = c.cfg.group, c.cfg.head_dim
    out, tau = o.out.double().cpu().numpy(), o.tau.double().cpu().numpy()
    Q = q.double().cpu().numpy()
    sc = scale if scale else d ** -0.5
    for b, n in enumerate(counts):
        seq = b if seq_ids is None else seq_ids[b]
        r0 = sum(counts[:b]) if start is None else start[b]
        fk = None if first_key is None else first_key[r0:r0 + n]
        for h in range(c.num_q_heads):
            if n == 0:
                continue
            K, V = dense(c, seq, h // G, "k"), dense(c, seq, h // G, "v")
            sl = 0.0 if slopes is None else float(slopes[h])
            ref, t, Pw, S = oq.attend(K, V, Q[r0:r0 + n, h], alpha, scale, softcap, sl, window,
                                      0 if prefix is None else prefix[b], fk)
            mag = (np.abs(Q[r0:r0 + n, h]) @ np.abs(K).T).max(initial=0.0) * sc
            delta = 2.0 ** -20 * (mag + sl * len(K) + softcap + 1.0)
            if alpha == 1.0:
                dp = 2 * delta * Pw
            else:
                beta, dz = 1.0 / (alpha - 1.0), 2 * (alpha - 1.0) * delta
                y = np.where(np.isfinite(S), S, -1e30) * (alpha - 1.0) - t[:, None]
                near = y > -dz
                dp = np.where(near, dz ** beta if beta < 1 else beta * np.maximum(y + dz, 0.0) ** (beta - 1) * dz, 0.0)
                dp = np.nan_to_num(dp)
                t_tol = 2 * (alpha - 1.0) * delta
            s = v_scales(c, seq, h // G)
            if alpha == 1.0:
                small = 2.0 ** -33 * (Pw * s).max(1, initial=0.0)[:, None] * np.isfinite(S)
            else:
                on = (Pw > 0) | (dp > 0)
                small = 2.0 ** -24 * Pw.max(1, initial=0.0)[:, None] * (on * s).max(1, initial=0.0)[:, None] * on
            tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 * Pw + small / s + dp) @ np.abs(V) + 1e-30
            err = np.abs(out[r0:r0 + n, h] - ref)
            assert np.all(err <= tol), (b, h, float((err / tol).max()))
            some = ~np.isnan(t)
            assert np.array_equal(np.isnan(tau[r0:r0 + n, h]), ~some), (b, h)
            if alpha == 1.0:
                t_tol = 2 * delta
            te = np.abs(tau[r0:r0 + n, h] - t)[some]
            assert np.all(te <= t_tol + 2.0 ** -23 * np.abs(t[some])), (b, h, te.max(initial=0.0), t_tol)
            assert not out[r0:r0 + n, h][~some].any()
