"""Differential attention, key weights and evictions as callers lay them out: rows that belong to nobody, queries that
are slices or broadcast, slots in any order, many slots, many KV heads, no statistic wanted, a pool that runs dry."""

import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

from q8_cases import batch_of, filled, i32
from test_q8_diff_gpu import check_diff, factors, gains
from test_q8_evict_gpu import check, make, spread_weights, state
from test_q8_weigh_gpu import check_weights, others_untouched, run, some_weights

pytestmark = pytest.mark.gpu

COUNTS = [[1, 0, 1, 1], [4, 2, 0, 3], [7, 0, 6, 1], [60, 9, 0, 33]]  # 8, 32, 56 and 480 rows with a group of 8


def laid_out(counts, order, total, gap):
    """Slots' first rows, the slots' rows lying in `order` with gaps before, between and behind them."""
    start, at = [0] * len(counts), gap
    for b in order:
        start[b] = at
        at += counts[b] + gap
    assert at <= total
    return start


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("code,d,P", [("int8", 64, 16), ("e4m3", 128, 32)])
def test_rows_of_nobody_and_slots_in_any_order(counts, code, d, P):
    """Sequences in other rows of the table than their slots, slots' rows out of order, and whatever lies between them:
    NaN in queries, statistics and factors of rows that belong to no slot."""
    g, seqs, order, gap = 8, [5, 1, 0, 3], [2, 0, 3, 1], 3
    lens = [300, 90, 40, 700, 1, 66]
    c, _ = filled(code, lens, [1], hkv=2, g=g, d=d, P=P, seed=3)
    n, total = sum(counts), sum(counts) + 5 * gap + 2
    start = laid_out(counts, order, total, gap)
    gen = torch.Generator(device="cuda").manual_seed(4)
    real = torch.randn(n, 2 * g, d, generator=gen, device="cuda").bfloat16()
    wide = torch.full((total, 2 * g + 3, d + 8), float("nan"), dtype=torch.bfloat16, device="cuda")  # slices of rows
    lam, coef = torch.full((total, g), float("nan"), device="cuda"), torch.full((total, 2 * g), float("nan"), device="cuda")
    lam_real = factors(n, g, True)
    coef_real = torch.rand(n, 2 * g, generator=gen, device="cuda")
    rows = torch.cat([torch.arange(start[b], start[b] + m) for b, m in enumerate(counts)]).cuda()
    wide[rows, 2:2 + 2 * g, :d], lam[rows], coef[rows] = real, lam_real, coef_real
    q = wide[:, 2:2 + 2 * g, :d]
    batch = B.Batch(i32(start), i32(counts), total, max(counts), i32(seqs))
    o = B.attend_diff_q8(c, q, lam, batch, gain=gains(d),
                         outputs=B.AttendOutputs(torch.full((total, g, d), 5.0, device="cuda").bfloat16(),
                                                 torch.full((total, 2 * g), float("nan"), device="cuda")))
    check_diff(c, real, counts, B.AttendOutputs(o.out[rows], o.tau[rows]), lam_real, gains(d), seq_ids=seqs)
    nobody = torch.ones(total, dtype=torch.bool, device="cuda")
    nobody[rows] = False
    assert bool((o.out[nobody] == 5.0).all()) and bool(o.tau[nobody].isnan().all())
    before = some_weights(c)
    after = B.weigh_q8(c, before.clone(), q, o.tau, batch, coef=coef, decay=1.5)
    check_weights(c, real, counts, o.tau[rows], before, after, coef=coef_real, decay=1.5, seq_ids=seqs)
    others_untouched(c, before, after, [s for s, m in zip(seqs, counts) if m])
    # the statistic is wanted by nobody
    alone = B.attend_diff_q8(c, q, lam, batch, gain=gains(d), outputs=B.AttendOutputs(torch.zeros_like(o.out), None))
    assert torch.equal(alone.out[rows], o.out[rows]) and c.device_status() == 0


@pytest.mark.parametrize("count", [1, 3, 50])
def test_broadcast_queries(count):
    """One row for all tokens and heads of a slot (strides of 0) answers as its copies do."""
    c, q = filled("int8", [400, 31], [count, count], hkv=2, g=4, d=128, P=32, seed=5)
    one = q[:1, :1].expand(2 * count, 8, 128)
    lam, batch = factors(2 * count, 4, False), batch_of([count] * 2)
    a, b = (B.attend_diff_q8(c, x, lam, batch) for x in (one, one.contiguous()))
    assert torch.equal(a.out, b.out) and torch.equal(a.tau, b.tau)
    wa, wb = (B.weigh_q8(c, B.alloc_weights(c), x, a.tau, batch) for x in (one, one.contiguous()))
    assert torch.equal(wa, wb) and bool(wa.any())


@pytest.mark.parametrize("n,count,g", [(600, 1, 2), (300, 5, 2), (300, 4, 8), (520, 3, 7), (300, 8, 6)])
def test_many_slots_of_each_variant(n, count, g):
    """More slots than a block keeps at hand, and than it has threads (512, or 256 for 17 to 32 rows a slot)."""
    counts = [0 if i % 11 == 5 else 1 + (i * 7) % count for i in range(n)]
    lens = [max(counts[i], 1) + (i * 13) % 50 for i in range(n)]
    c, q = filled("int8", lens, counts, hkv=1, g=g, d=64, P=16, seed=6)
    run(c, q, counts, decay=0.5)
    lam = factors(sum(counts), g // 2, True)
    if g % 2 == 0:
        check_diff(c, q, counts, B.attend_diff_q8(c, q, lam, batch_of(counts)), lam)
    assert c.device_status() == 0


@pytest.mark.parametrize("hkv,g", [(96, 2), (300, 1)])
def test_many_kv_heads(hkv, g):
    lens, counts = [70, 200], [1, 1]
    c, q = filled("e4m3", lens, counts, hkv=hkv, g=g, d=64, P=16, seed=7)
    run(c, q, counts)
    run(c, torch.randn(80, hkv * g, 64, device="cuda").bfloat16(), [40, 40])
    if g == 2:
        lam = factors(2, hkv, False)
        check_diff(c, q, counts, B.attend_diff_q8(c, q, lam, batch_of(counts)), lam)
    c, pool = make("int8", lens, hkv=hkv, d=64, P=16, seed=8)
    check(c, pool, spread_weights(c), "int8", [1, 0], 50, sinks=1, recent=7)


def test_a_pool_that_runs_dry_under_a_budget():
    """Slots are refused while no page is left, and admitted again behind evictions; what is refused is neither weighed
    nor evicted."""
    hkv, g, d, P = 1, 2, 64, 16
    c, pool = B.QuantCache(hkv, g, d, P, 3, 8, 7, torch.int8), B.PagePool.full(7)
    step = B.QuantStep(c, pool, 3, 20, budget=B.KeyBudget(16, above=40, sinks=1, recent=4))
    gen = torch.Generator(device="cuda").manual_seed(9)
    L, refused = [0, 0, 0], 0
    for i in range(14):
        counts = [20, 20, 20] if i % 2 == 0 else [0, 20, 3]
        free = int(pool.free_count)
        want, stop = [], False
        for b in range(3):  # in order, the first that does not fit stops those behind it
            need = -(-(L[b] + counts[b]) // P) - -(-L[b] // P)
            free -= need
            stop = stop or free < 0
            want.append(0 if stop else counts[b])
        before = state(c, pool, step.budget.weights)
        x = torch.randn(sum(counts), 4 * hkv, d, generator=gen, device="cuda").bfloat16()
        step.run(i32(counts), i32([0, 1, 2]), x[:, :2], x[:, 2:3], x[:, 3:])
        torch.cuda.synchronize()
        assert step.plan.count.tolist() == want
        L = [n + m for n, m in zip(L, want)]
        L = [16 if n > 40 and m else n for n, m in zip(L, want)]
        assert c.seq_lens.tolist() == L
        assert int(pool.free_count) == 7 - sum(-(-n // P) for n in L)
        assert c.device_status() in (0, B.DEV_CAPACITY)
        c.status.zero_()
        refused += want != counts
        for b in range(3):
            if want[b] == 0 and L[b]:
                ph = c.block_table[b, :-(-L[b] // P)].long()
                assert torch.equal(before["w"][ph], step.budget.weights[ph])
    held = [p for b in range(3) for p in c.block_table[b, :-(-L[b] // P)].tolist()]
    assert refused > 2 and sorted(held + pool.free_pages[:int(pool.free_count)].tolist()) == list(range(7))
