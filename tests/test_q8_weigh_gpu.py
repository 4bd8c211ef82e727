"""The weight that rows give to the keys of the 8-bit cache, against the oracle."""

import numpy as np
import pytest
import torch

from oracle import q8 as oq
from sparse_entmax_attention_gb300 import binding as B

from q8_cases import batch_of, dense, filled, i32

pytestmark = pytest.mark.gpu


def rows_of(c, w, seq, h):
    """[L] weights of one sequence's keys."""
    P, L = c.cfg.page_size, int(c.seq_lens[seq])
    return w[c.block_table[seq, :-(-L // P)].long(), h].reshape(-1)[:L].double().cpu().numpy()


def check_weights(c, q, counts, tau, before, after, alpha=1.0, coef=None, decay=1.0, fresh=None, seq_ids=None,
                  scale=0.0, softcap=0.0, slopes=None, window=0, prefix=None, first_key=None):
    """A score is off by at most δ = 2^-20·(Σ|q||k|·scale + slope·L + cap + 1) (as for attention), the statistic's change
    to base 2 by 2^-23·|tau|, an exponential by 2^-21: a softmax weight by p·(2δ + 2^-22·|tau| + 2^-20). An entmax
    weight y^β moves by at most β·(y+η)^{β−1}·η for β ≥ 1 and η^β below, η = (α−1)·(δ + 2^-23·|tau|), and its
    power's own error is β·2^-21. A sum of n terms: 2^-24·(n + 4) of the sum of their sizes."""
    G, d = c.cfg.group, c.cfg.head_dim
    Q, T = q.double().cpu().numpy(), tau.double().cpu().numpy()
    C = np.ones_like(T) if coef is None else coef.double().cpu().numpy()
    C = np.where(C > 0, C, 0.0)
    sc = scale if scale else d ** -0.5
    for b, n in enumerate(counts):
        if n == 0:
            continue
        seq = b if seq_ids is None else seq_ids[b]
        r0, L = sum(counts[:b]), int(c.seq_lens[seq])
        fk = None if first_key is None else first_key[r0:r0 + n]
        new = min(max(n if fresh is None else fresh[b], 0), L)
        for h in range(c.cfg.num_kv_heads):
            K = dense(c, seq, h, "k")
            old = rows_of(c, before, seq, h)
            old = np.where(np.arange(L) < L - new, old * np.float64(np.float32(decay)) if decay else 0.0, 0.0)
            want, tol = old.copy(), 2.0 ** -24 * np.abs(old)
            for hd in range(h * G, h * G + G):
                x = Q[r0:r0 + n, hd]
                sl = 0.0 if slopes is None else float(slopes[hd])
                _, _, _, S = oq.attend(K, K, x, 1.0, scale, softcap, sl, window, 0 if prefix is None else prefix[b], fk)
                t = T[r0:r0 + n, hd]
                p = oq.key_weights(S, t, alpha)
                t = np.abs(np.where(np.isfinite(t), t, 0.0))[:, None]
                mag = (np.abs(x) @ np.abs(K).T) * sc
                delta = 2.0 ** -20 * (mag + sl * L + softcap + 1.0)
                if alpha == 1.0:
                    dp = p * np.expm1(2 * delta + 2.0 ** -22 * t + 2.0 ** -20)
                else:
                    beta, eta = 1.0 / (alpha - 1.0), (alpha - 1.0) * (delta + 2.0 ** -23 * t)
                    y = np.where(np.isfinite(S), S, -1e30) * (alpha - 1.0) - np.where(np.isfinite(T[r0:r0 + n, hd]), T[r0:r0 + n, hd], 1e30)[:, None]
                    dp = np.where(y > -eta, eta ** beta if beta < 1 else beta * np.maximum(y + eta, 0.0) ** (beta - 1) * eta, 0.0)
                    dp = dp + p * beta * 2.0 ** -21
                k = C[r0:r0 + n, hd][:, None]
                want += (k * p).sum(0)
                tol += (k * dp).sum(0)
            tol += 2.0 ** -24 * (n * G + 4) * np.abs(want) + 1e-35
            got = rows_of(c, after, seq, h)
            assert np.all(np.abs(got - want) <= tol), (b, h, float((np.abs(got - want) / tol).max()))


def some_weights(c, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.exp(torch.randn(B.alloc_weights(c).shape, generator=gen, device="cuda"))


def others_untouched(c, before, after, seqs):
    """Places of no key of these sequences keep their bits."""
    mark = torch.zeros(before.shape, dtype=torch.bool, device="cuda")
    P = c.cfg.page_size
    for s in seqs:
        L = int(c.seq_lens[s])
        for j in range(-(-L // P)):
            mark[int(c.block_table[s, j]), :, :min(P, L - j * P)] = True
    assert torch.equal(before[~mark], after[~mark])


def run(c, q, counts, alpha=1.0, seq_ids=None, seed=0, tau=None, **kw):
    """Attention for the statistic, then the weights; everything checked."""
    score = {k: v for k, v in kw.items() if k in ("scale", "softcap", "slopes", "window", "prefix", "first_key")}
    on = {k: i32(v) if k in ("prefix", "first_key", "fresh") else v for k, v in kw.items()}
    batch = batch_of(counts, seq_ids)
    if tau is None:
        tau = B.attend_q8(c, q, batch, alpha=alpha, **{k: on[k] for k in score}).tau
    before = some_weights(c, seed)
    after = before.clone()
    assert B.weigh_q8(c, after, q, tau, batch, alpha=alpha, **on) is after
    torch.cuda.synchronize()
    assert c.device_status() == 0
    check_weights(c, q, counts, tau, before, after, alpha, seq_ids=seq_ids, **kw)
    used = [(b if seq_ids is None else seq_ids[b]) for b, n in enumerate(counts) if n]
    others_untouched(c, before, after, used)
    return before, after


@pytest.mark.parametrize("code,d,P", [("int8", 128, 32), ("e4m3", 128, 16), ("int8", 64, 16), ("e4m3", 64, 32)])
@pytest.mark.parametrize("g,alpha", [(1, 1.0), (3, 1.0), (8, 1.0), (4, 1.5), (5, 2.0), (2, 1.25), (4, 3.0)])
def test_single_rows(code, d, P, g, alpha):
    lens = [1, 2, 33, 700, 5001]
    c, q = filled(code, lens, [1] * 5, hkv=2, g=g, d=d, P=P, seed=g)
    run(c, q, [1] * 5, alpha)
    run(c, q, [1] * 5, alpha, decay=0.75, window=100, softcap=15.0)


@pytest.mark.parametrize("code,d,P,g,counts", [
    ("int8", 128, 32, 4, [3, 1, 0, 2]), ("e4m3", 64, 16, 5, [3, 2, 1, 3]), ("int8", 128, 16, 4, [9, 8, 3, 1]),
    ("int8", 128, 16, 4, [70, 1, 130, 33]), ("e4m3", 128, 32, 3, [90, 0, 43, 20]), ("e4m3", 64, 16, 7, [200, 129, 1, 64]),
    ("int8", 64, 32, 8, [17, 300, 2, 1])])
def test_several_rows_with_masks(code, d, P, g, counts):
    lens = [max(1, n + x) for n, x in zip(counts, (500, 3, 1000, 0))]
    c, q = filled(code, lens, counts, hkv=2, g=g, d=d, P=P, seed=7)
    total, Hq = sum(counts), 2 * g
    first = [(L - n + i if i % 5 else L) if i % 3 == 2 else max(0, L - n + i - 40)
             for L, n in zip(lens, counts) for i in range(n)]
    slopes = torch.exp2(-torch.arange(1, Hq + 1, device="cuda").float())
    gen = torch.Generator(device="cuda").manual_seed(2)
    coef = torch.randn(total, Hq, generator=gen, device="cuda")   # half of them do not count
    coef[0, 0] = float("nan")
    for kw in ({}, {"softcap": 20.0, "window": 90, "decay": 0.5}, {"prefix": [30, 0, 5, 2], "window": 8},
               {"first_key": first, "fresh": [100, 2000, 0, 1]}, {"slopes": slopes, "softcap": 8.0, "coef": coef},
               {"decay": 0.0, "fresh": [0, 0, 0, 0], "scale": 0.01}):
        run(c, q, counts, **kw)


def test_rows_without_a_statistic_add_nothing():
    for counts in ([2, 1], [40, 3]):
        c, q = filled("int8", [300, 50], counts, hkv=2, g=4, d=128, P=32)
        tau = B.attend_q8(c, q, batch_of(counts)).tau
        tau[0, 1], tau[1, 2], tau[2, 3] = float("nan"), float("inf"), -float("inf")
        q = q.clone()
        q[0, 1], q[1, 2, 7] = float("nan"), float("inf")
        before = some_weights(c)
        after = before.clone()
        B.weigh_q8(c, after, q, tau, batch_of(counts))
        q[0, 1], q[1, 2, 7] = 0.0, 0.0
        check_weights(c, q, counts, tau, before, after)


def test_weights_that_are_not_read_may_be_anything():
    for counts, kw in (([1, 1], {"decay": 0.0}), ([30, 2], {"decay": 0.0}), ([30, 2], {"fresh": [300, 50]})):
        c, q = filled("e4m3", [300, 50], counts, hkv=2, g=4, d=64, P=16)
        tau = B.attend_q8(c, q, batch_of(counts)).tau
        after = torch.full_like(B.alloc_weights(c), float("nan"))
        B.weigh_q8(c, after, q, tau, batch_of(counts), **{k: i32(v) if k == "fresh" else v for k, v in kw.items()})
        check_weights(c, q, counts, tau, torch.ones_like(after), after, **kw)


@pytest.mark.parametrize("n,count,g,alpha", [(70000, 1, 2, 1.0), (70000, 1, 4, 1.5), (40000, 60, 2, 1.0), (9000, 9000, 1, 1.0)])
def test_long_sequences(n, count, g, alpha):
    """Each row's weights add up to one: the keys' sum is the count of rows and heads."""
    c, q = filled("int8", [n], [count], hkv=1, g=g, d=64, P=32, seed=3)
    tau = B.attend_q8(c, q, batch_of([count]), alpha=alpha).tau
    w = B.alloc_weights(c)
    B.weigh_q8(c, w, q, tau, batch_of([count]), alpha=alpha)
    got = float(torch.from_numpy(rows_of(c, w, 0, 0)).sum())
    # (softmax: a weight is good to 2^-20·(Σ|q||k|/8 + |tau| + 2), here below 2^-13; entmax: the threshold's sum to 2^-14 + 2^-20)
    assert abs(got - count * g) <= 2.0 ** -13 * count * g
    if count < 100:
        run(c, q, [count], alpha)


def test_a_bad_page_is_flagged_and_skipped():
    for counts in ([1], [40]):
        c, q = filled("int8", [100], counts, hkv=1, g=2, d=64, P=16)
        tau = B.attend_q8(c, q, batch_of(counts)).tau
        page = int(c.block_table[0, 2])
        c.block_table[0, 2] = -5
        before = some_weights(c)
        after = before.clone()
        B.weigh_q8(c, after, q, tau, batch_of(counts))
        assert c.device_status() == B.DEV_BAD_PAGE_TABLE
        assert torch.equal(before[page], after[page])
        c.block_table[0, 2] = page
        lost = before.clone()
        B.weigh_q8(c, lost, q, tau, batch_of(counts))
        lost[page] = before[page]
        assert torch.equal(lost, after)


def test_bad_slots_are_left_as_they_were():
    c, q = filled("int8", [100, 80, 60], [2, 2, 2], hkv=2, g=2, d=64, P=16)
    tau = B.attend_q8(c, q, batch_of([2, 2, 2])).tau
    before = some_weights(c)
    after = before.clone()
    B.weigh_q8(c, after, q, tau, B.Batch(i32([0, 2, 4]), i32([2, 90, 2]), 6, 2, i32([0, 1, 9])))
    assert c.device_status() == B.DEV_BAD_BATCH | B.DEV_BAD_SEQ_ID
    check_weights(c, q[:2], [2], tau[:2], before, after, seq_ids=[0])
    others_untouched(c, before, after, [0])


def test_equal_calls_give_equal_bits_captured_or_not():
    for counts in ([1, 1, 1], [50, 3, 200]):
        c, q = filled("e4m3", [3000, 10, 900], counts, hkv=2, g=4, d=128, P=16)
        batch = batch_of(counts)
        tau = B.attend_q8(c, q, batch).tau
        before = some_weights(c)
        want = B.weigh_q8(c, before.clone(), q, tau, batch, decay=0.9)
        ws, w = B.alloc_weigh_workspace(c, batch), before.clone()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        B.weigh_q8(c, w, q, tau, batch, decay=0.9, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(w, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.weigh_q8(c, w, q, tau, batch, decay=0.9, workspace=ws)
        for _ in range(3):
            w.copy_(before)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(w, want)


def test_more_slots_than_a_block_keeps_at_hand():
    n = 300
    c, q = filled("int8", [5 + i % 40 for i in range(n)], [1] * n, hkv=1, g=2, d=64, P=16)
    run(c, q, [1] * n)
    c, q = filled("int8", [20 + i % 40 for i in range(n)], [9 + i % 9 for i in range(n)], hkv=1, g=4, d=64, P=16)
    run(c, q, [9 + i % 9 for i in range(n)], decay=0.5)


def test_more_slots_than_a_round_of_the_planning():
    n = 1100
    counts = [5 + i % 7 if i % 5 else 0 for i in range(n)]
    c, q = filled("int8", [12 + i % 30 for i in range(n)], counts, hkv=1, g=4, d=64, P=16)
    run(c, q, counts)


def test_slots_that_claim_the_same_rows_stop_at_the_lists_end():
    """The third slot's row tiles do not fit the list that the rows have room for: it is flagged and left."""
    c, q = filled("int8", [90, 80, 70], [60, 0, 0], hkv=1, g=8, d=64, P=16)
    tau = B.attend_q8(c, q, batch_of([60])).tau
    before = some_weights(c)
    after = before.clone()
    B.weigh_q8(c, after, q, tau, B.Batch(i32([0, 0, 0]), i32([60, 60, 60]), 60, 60))
    assert c.device_status() == B.DEV_BAD_BATCH
    check_weights(c, q, [60], tau, before, after)
    others_untouched(c, before, after, [0, 1])
    assert not torch.equal(before, after)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_rows_of_unlike_loudness_share_a_tile(code, softcap):
    """Queries over 24 factors of two in one tile, tiles of nothing but tiny or zero queries, and rows that add nothing
    with infinities, NaN and huge values in them."""
    counts = [100, 64, 40]
    c, q = filled(code, [900, 300, 500], counts, hkv=2, g=4, d=128, P=32, seed=8)
    q = q.clone()
    for t in range(100):
        q[t] *= 2.0 ** (4 - t % 25)
    q[100:132] *= 2.0 ** -100
    q[132:164] = 0.0
    tau = B.attend_q8(c, q, batch_of(counts), softcap=softcap).tau.clone()
    loud = q.clone()
    for t, bad in ((3, 1e38), (50, float("inf")), (99, float("nan")), (170, -1e30)):
        loud[t, ::3] = bad
        q[t, ::3] = 0.0
        tau[t, ::3] = float("nan")
    before = some_weights(c)
    after = before.clone()
    B.weigh_q8(c, after, loud, tau, batch_of(counts), softcap=softcap, decay=0.5)
    check_weights(c, q, counts, tau, before, after, decay=0.5, softcap=softcap)
    plain = before.clone()
    B.weigh_q8(c, plain, q, tau, batch_of(counts), softcap=softcap, decay=0.5)
    assert torch.equal(plain, after) and c.device_status() == 0
