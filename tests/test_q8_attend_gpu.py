"""Attention over the 8-bit cache against the float64 oracle."""

import math

import numpy as np
import pytest
import torch

from oracle import entmax as em
from sparse_entmax_attention_gb300 import binding as B

from q8_cases import batch_of, check_attend, dense, empty_cache, filled, i32, v_scales

pytestmark = pytest.mark.gpu


def run(code, lens, counts, alpha=1.0, seed=0, cache_kw=None, **score):
    c, q = filled(code, lens, counts, seed=seed, **(cache_kw or {}))
    dev = dict(score)
    if score.get("slopes") is not None:
        dev["slopes"] = torch.tensor(score["slopes"], dtype=torch.float32, device="cuda")
    for k in ("prefix", "first_key"):
        if score.get(k) is not None:
            dev[k] = i32(score[k])
    o = B.attend_q8(c, q, batch_of(counts), alpha=alpha, **dev)
    torch.cuda.synchronize()
    assert c.device_status() == 0
    check_attend(c, q, counts, o, alpha=alpha, **score)
    return c, q, o


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d,P", [(128, 32), (128, 16), (64, 32), (64, 16)])
@pytest.mark.parametrize("alpha", [1.0, 1.5, 2.0])
def test_single_tokens(code, d, P, alpha):
    lens = [1, 2, P - 1, P, P + 1, 333, 1500]
    run(code, lens, [1] * len(lens), alpha=alpha, cache_kw=dict(d=d, P=P))


@pytest.mark.parametrize("g", [1, 2, 3, 5, 6, 7, 8])
@pytest.mark.parametrize("alpha", [1.0, 1.5])
def test_groups(g, alpha):
    run("int8", [70, 5], [1, 1], alpha=alpha, cache_kw=dict(hkv=3, g=g, d=64, P=16))
    if alpha == 1.0:
        run("e4m3", [70, 5], [3, 2], cache_kw=dict(hkv=3, g=g, d=64, P=16))


FORMS = [dict(softcap=5.0), dict(slopes="yes"), dict(window=1), dict(window=40), dict(prefix=[0, 17, 900, 1]),
         dict(window=20, prefix=[40, 40, 2, 33]), dict(first_key="yes"), dict(scale=0.5),
         dict(softcap=20.0, slopes="yes", window=100, prefix=[3, 200, 0, 50], first_key="yes")]


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "+".join(f))
@pytest.mark.parametrize("counts,alpha", [([1, 1, 1, 1], 1.0), ([1, 1, 1, 1], 1.5), ([2, 1, 4, 3], 1.0),
                                          ([37, 1, 130, 3], 1.0)])
def test_score_forms_and_masks(form, counts, alpha):
    lens = [40, 200, 700, 65]
    form = dict(form)
    if form.get("slopes"):
        form["slopes"] = [0.0, 0.5, 2.0 ** -6, 0.1, 1.0, 0.0, 0.003, 0.25]
    if form.get("first_key"):
        # a document's start, the row's own position, and one behind it: a row that sees nothing
        form["first_key"] = [lens[b] - counts[b] + i - (25, 0, 90, -1)[(b + i) % 4]
                             for b in range(4) for i in range(counts[b])]
    run("int8", lens, counts, alpha=alpha, **form)


@pytest.mark.parametrize("counts", [[5, 0, 1], [16, 17, 2], [64, 100, 33], [129, 1, 300]])
@pytest.mark.parametrize("code,d,P,g", [("int8", 128, 32, 4), ("e4m3", 128, 16, 4), ("e4m3", 64, 32, 8),
                                        ("int8", 64, 16, 3)])
def test_several_new_tokens(counts, code, d, P, g):
    lens = [n + m for n, m in zip((0, 50, 301), counts)]
    run(code, lens, counts, cache_kw=dict(d=d, P=P, g=g), softcap=8.0)


def test_rows_without_keys_and_garbage_behind_the_end():
    """Codes behind the last token are NaN patterns or -128, stale scales NaN: none is seen."""
    for code in ("int8", "e4m3"):
        for alpha in (1.0, 1.5):
            lens, counts = [1, 19, 40], [1, 1, 1]
            c, q = filled(code, lens, counts, garbage=True, P=16, d=64)
            fk = i32([5, 0, 40])
            o = B.attend_q8(c, q, batch_of(counts), alpha=alpha, first_key=fk)
            check_attend(c, q, counts, o, alpha=alpha, first_key=[5, 0, 40])
            assert torch.isnan(o.tau[0]).all() and torch.isnan(o.tau[2]).all() and not torch.isnan(o.tau[1]).any()
    counts = [70, 41, 33]
    lens = [70, 77, 40]
    c, q = filled("e4m3", lens, counts, garbage=True, P=16, d=64)
    o = B.attend_q8(c, q, batch_of(counts))
    check_attend(c, q, counts, o)


@pytest.mark.parametrize("counts", [[1, 1, 0, 1], [3, 2, 0, 4], [90, 2, 0, 140]])
def test_idle_and_refused_slots_leave_their_rows(counts):
    lens = [200, 100, 50, 300]
    seqs = [1, 3, 77, 0]  # the idle slot's row is not looked at
    lens_by = [lens[3], lens[0], 10, lens[1]]
    c, _ = filled("int8", lens_by, [1], hkv=2, g=4)
    batch = batch_of(counts, seqs, gap=2)
    q = torch.randn(batch.total, 8, 128, device="cuda").bfloat16()
    o = B.alloc_attend_outputs(c, batch)
    o.out.fill_(9.0)
    o.tau.fill_(9.0)
    B.attend_q8(c, q, batch, outputs=o)
    start = batch.start.tolist()
    check_attend(c, q, counts, o, seq_ids=seqs, start=start)
    own = torch.zeros(batch.total, dtype=torch.bool)
    for s0, n in zip(start, counts):
        own[s0:s0 + n] = True
    assert bool((o.out[~own.cuda()] == 9.0).all()) and bool((o.tau[~own.cuda()] == 9.0).all())
    assert c.device_status() == 0
    # more rows than the sequence has tokens, rows outside the arrays, a bad sequence
    o.out.fill_(9.0)
    bad = B.Batch(i32([0, batch.total, 0]), i32([11, 1, 1]), batch.total, 11, i32([2, 1, 9]))
    B.attend_q8(c, q, bad, outputs=o)
    assert bool((o.out == 9.0).all()) and c.device_status() == B.DEV_BAD_BATCH | B.DEV_BAD_SEQ_ID


@pytest.mark.parametrize("alpha,n", [(1.0, 1), (1.5, 1), (1.0, 40)])
def test_bad_page_entries_are_flagged_and_skipped(alpha, n):
    c, q = filled("int8", [200], [n], P=32)
    c.block_table[0, 2] = 10 ** 6
    batch = batch_of([n])
    o = B.attend_q8(c, q, batch, alpha=alpha)
    assert c.device_status() == B.DEV_BAD_PAGE_TABLE
    # as if that page's keys were masked: the same cache without it
    c2, _ = filled("int8", [200], [n], P=32)
    keep = [j for j in range(200) if not 64 <= j < 96]
    K, V = dense(c2, 0, 0, "k"), dense(c2, 0, 0, "v")
    Q = q.double().cpu().numpy()[:, 0]
    for i in (0, n - 1):
        pos = 200 - n + i
        idx = [j for j in keep if j <= pos]
        s = K[idx] @ Q[i] / math.sqrt(128)
        p, t = em.softmax(s) if alpha == 1.0 else em.entmax(s, alpha)
        assert abs(float(o.tau[i, 0]) - t) < 1e-4
        assert np.abs(o.out[i, 0].double().cpu().numpy() - p @ V[idx]).max() < 2.0 ** -6 * np.abs(V).max()


@pytest.mark.parametrize("alpha", [1.25, 1.5, 2.0, 3.0])
@pytest.mark.parametrize("kind", ["flat", "one", "plain"])
def test_entmax_supports(alpha, kind):
    """Every key in the support (equal keys), a single one, and what random keys give."""
    lens = [3000, 1, 77]
    c, q = filled("int8", lens, [1, 1, 1], P=16, d=64, loud=1.0 if kind != "one" else 30.0)
    if kind == "flat":
        k = torch.ones(sum(lens), 2, 64, device="cuda").bfloat16()
        v = torch.randn(sum(lens), 2, 64, device="cuda").bfloat16()
        B.append_q8(c, k, v, batch_of(lens))
    o = B.attend_q8(c, q, batch_of([1, 1, 1]), alpha=alpha)
    assert c.device_status() == 0
    check_attend(c, q, [1, 1, 1], o, alpha=alpha)


@pytest.mark.parametrize("alpha,n,L", [(1.0, 1, 70000), (1.5, 1, 70000), (1.0, 3, 33000), (1.0, 200, 9000)])
def test_long_sequences_beside_short_ones(alpha, n, L):
    lens = [n, L, n + 3]
    run("int8", lens, [n] * 3, alpha=alpha, cache_kw=dict(hkv=1, g=2, P=16))


def test_a_strong_key_does_not_drown_many_weak_ones():
    """One key with weight 1 and 60000 with 2^-22 each: together they are 1.4% of the output."""
    L, d = 60000, 64
    c = empty_cache("int8", [L], hkv=1, g=1, d=d, P=32)
    k = torch.zeros(L, 1, d, device="cuda")
    k[:, 0, 0] = -1.0
    k[100, 0, 0] = 1.0
    v = torch.ones(L, 1, d, device="cuda")
    v[100] = 0
    B.append_q8(c, k.bfloat16(), v.bfloat16(), batch_of([L]))
    for n in (1, 150):
        q = torch.zeros(n, 1, d, device="cuda")
        q[:, 0, 0] = 22 * math.log(2.0) / 2 * math.sqrt(d)
        o = B.attend_q8(c, q.bfloat16(), batch_of([n]))
        check_attend(c, q.bfloat16(), [n], o)


@pytest.mark.parametrize("alpha,counts", [(1.0, [1, 1]), (1.5, [1, 1]), (1.0, [4, 3]), (1.0, [140, 90])])
def test_equal_calls_give_equal_bits_on_any_stream(alpha, counts):
    c, q = filled("e4m3", [3000, 500], counts)
    batch = batch_of(counts)
    ws = B.alloc_attend_workspace(c, batch, alpha)
    first = B.attend_q8(c, q, batch, alpha=alpha, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws2 = B.alloc_attend_workspace(c, batch, alpha)
    ws2.fill_(0xff)  # contents of the workspace do not matter
    o2 = B.alloc_attend_outputs(c, batch)
    torch.cuda.synchronize()
    for _ in range(3):
        B.attend_q8(c, q, batch, alpha=alpha, workspace=ws2, outputs=o2, stream=side)
        side.synchronize()
        assert torch.equal(first.out, o2.out) and torch.equal(first.tau, o2.tau)


def test_strided_queries_and_outputs():
    c, _ = filled("int8", [300, 80], [1], g=4)
    for counts in ([1, 1], [5, 2], [100, 60]):
        total = sum(counts)
        qkv = torch.randn(total, 12, 128, device="cuda").bfloat16()
        out = torch.zeros(total, 3, 8, 128, dtype=torch.bfloat16, device="cuda")
        o = B.AttendOutputs(out[:, 1], torch.zeros(total, 8, device="cuda"))
        B.attend_q8(c, qkv[:, :8], batch_of(counts), outputs=o)
        check_attend(c, qkv[:, :8], counts, o)
        assert not out[:, 0].any() and not out[:, 2].any()


def test_infinite_and_huge_queries():
    """A row of large queries is exact up to its range; a non-finite one spoils its own rows only."""
    c, q = filled("int8", [100, 100], [1, 1], g=2)
    q2 = q.clone()
    q2[0] *= 2.0 ** 100
    o = B.attend_q8(c, q2, batch_of([1, 1]), scale=2.0 ** -103)
    o1 = B.attend_q8(c, q, batch_of([1, 1]), scale=2.0 ** -3)
    assert torch.equal(o.out[0], o1.out[0])
    q2[0, 0, 3] = float("nan")
    base = B.attend_q8(c, q, batch_of([1, 1]))
    o = B.attend_q8(c, q2, batch_of([1, 1]))
    assert torch.isnan(o.out[0, 0]).all() and torch.equal(o.out[1], base.out[1])


@pytest.mark.parametrize("code,alpha,most", [("int8", 1.0, 1), ("e4m3", 1.0, 3), ("int8", 1.5, 1), ("int8", 1.0, 20)])
@pytest.mark.parametrize("n", [300, 1100])
def test_many_slots(code, alpha, most, n):
    """More slots than any kernel keeps in shared memory or lists at once, some of them idle."""
    lens = [1 + (b * 7) % 45 + most for b in range(n)]
    counts = [(b * 5) % (most + 1) if most > 1 else int(b % 9 != 4) for b in range(n)]
    run(code, lens, counts, alpha=alpha, cache_kw=dict(hkv=1, g=4, d=64, P=16))


def test_many_tiles_a_block():
    """Pieces of more than 32 tiles, over several items: sampled rows against the oracle."""
    L, n, hkv, g = 9500, 1100, 8, 4
    c, q = filled("int8", [L, 300], [n, 300], hkv=hkv, g=g)
    o = B.attend_q8(c, q, batch_of([n, 300]), softcap=6.0, window=9000)
    assert c.device_status() == 0
    rows = [0, 1, 63, 64, 500, 767, n - 1]
    for h in (0, 13, 31):
        K, V = dense(c, 0, h // g, "k"), dense(c, 0, h // g, "v")
        Q = q[:n, h].double().cpu().numpy()
        for i in rows:
            at = L - n + i  # keys at - 8999 .. at of this row
            lo = max(0, at - 8999)
            s = 6.0 * np.tanh(K[lo:at + 1] @ Q[i] / math.sqrt(128) / 6.0)
            p, t = em.softmax(s)
            delta = 2.0 ** -20 * ((np.abs(K[lo:at + 1]) @ np.abs(Q[i])).max() / math.sqrt(128) + 7.0)
            sc = v_scales(c, 0, h // g)[lo:at + 1]
            tol = (2.0 ** -8 * np.abs(p @ V[lo:at + 1])
                   + ((2.0 ** -11 + 2 * delta) * p + 2.0 ** -33 * (p * sc).max() / sc) @ np.abs(V[lo:at + 1]))
            assert np.all(np.abs(o.out[i, h].double().cpu().numpy() - p @ V[lo:at + 1]) <= tol), (h, i)
            assert abs(float(o.tau[i, h]) - t) <= 2 * delta + 2.0 ** -23 * abs(t)


@pytest.mark.parametrize("counts,alpha", [([1, 1], 1.0), ([1, 1], 1.5), ([6, 2], 1.0), ([90, 40], 1.0)])
def test_pages_beyond_32_bit_offsets(counts, alpha):
    """The same tokens in a small pool and in the last pages of one of 4.9 GB a side."""
    lens = [500, 210]
    small, q = filled("int8", lens, counts, hkv=8, g=4)
    n, P = 150000, 32
    big = B.QuantCache(8, 4, 128, P, 2, 17, n, torch.int8)
    big.block_table.copy_(n - 1 - small.block_table)
    big.seq_lens.copy_(small.seq_lens)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(sum(lens), 8, 128, generator=gen, device="cuda").bfloat16()
    v = torch.randn(sum(lens), 8, 128, generator=gen, device="cuda").bfloat16()
    B.append_q8(big, k, v, batch_of(lens))
    at = [i32([0, 0])] * 2
    back = [B.read_q8(c, f, batch_of(lens)) for c, f in zip((small, big), at)]
    assert torch.equal(back[0][0], back[1][0]) and torch.equal(back[0][1], back[1][1])
    a, b = (B.attend_q8(c, q, batch_of(counts), alpha=alpha) for c in (small, big))
    assert big.device_status() == 0
    assert torch.equal(a.out, b.out) and torch.equal(a.tau, b.tau)


def test_rows_claimed_by_several_slots_are_flagged():
    """More items than the rows allow: the call ends, and says so."""
    c, _ = filled("int8", [600, 600, 600, 600], [1], hkv=1, g=8)
    start, count = i32([0] * 4), i32([600] * 4)
    q = torch.randn(600, 8, 128, device="cuda").bfloat16()
    B.attend_q8(c, q, B.Batch(start, count, 600, 600))
    assert c.device_status() == B.DEV_BAD_BATCH


@pytest.mark.parametrize("blind", [[2], [0, 2], [1], [0, 1, 2]])
def test_chunks_whose_rows_see_nothing(blind):
    """Slots without a visible key, last ones among them, beside others, over several KV heads."""
    lens, counts = [700, 2100, 300], [100, 310, 90]
    fk = [10 ** 6 if b in blind else 0 for b in range(3) for _ in range(counts[b])]
    _, _, o = run("int8", lens, counts, cache_kw=dict(hkv=8, g=4, d=64, P=16), first_key=fk)
    for b in blind:
        at = sum(counts[:b])
        assert torch.isnan(o.tau[at:at + counts[b]]).all() and not o.out[at:at + counts[b]].any()
