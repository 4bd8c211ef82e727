"""Sequences held to a budget of keys: plan, append, attend (differential too),
weigh and evict in one captured step, against the same calls one by one and the
oracle."""

import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

from q8_cases import DT, check_attend, i32
from test_q8_diff_gpu import check_diff, factors, gains
from test_q8_evict_gpu import expect, same, state
from test_q8_weigh_gpu import check_weights

pytestmark = pytest.mark.gpu


def rows(seed, counts, hkv, g, d):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(sum(counts), (g + 2) * hkv, d, generator=gen, device="cuda").bfloat16()
    return qkv[:, :g * hkv], qkv[:, g * hkv:g * hkv + hkv], qkv[:, g * hkv + hkv:]


@pytest.mark.parametrize("code,most,alpha,diff", [("int8", 1, 1.0, True), ("e4m3", 1, 1.5, False), ("int8", 40, 1.0, False),
                                                  ("e4m3", 40, 1.0, True)])
def test_captured_step_matches_eager_calls_and_the_oracle(code, most, alpha, diff):
    hkv, g, d, P, slots, n_rows, pages = 2, 4, 64, 16, 4, 6, 40
    caches = [B.QuantCache(hkv, g, d, P, n_rows, 30, pages, DT[code]) for _ in range(2)]
    pools = [B.PagePool.full(pages) for _ in range(2)]
    lam, gain = (factors(1, g, False), gains(d)) if diff else (None, None)
    keep, above, sinks, recent, decay = (20, 24, 2, 6, 0.9) if most == 1 else (60, 60, 4, 30, 1.0)
    budget = B.KeyBudget(keep, above, sinks, recent, decay)
    score = dict(softcap=12.0)
    step = B.QuantStep(caches[1], pools[1], slots, most, alpha=alpha, lam=lam, gain=gain, budget=budget, **score)
    w = B.alloc_weights(caches[0])
    # growing sequences, idle slots with ids of nobody, a sequence that leaves, and one in its place
    runs = [([most] * 4, [0, 1, 2, 3])] * 3 + [([1, 0, most, 1], [0, 99, 2, 3]), ("release", [1])]
    runs += [([1, most, 1, 0], [0, 1, 5, 0])] * (30 if most == 1 else 4)
    for i, (counts, seqs) in enumerate(runs):
        if counts == "release":
            for c, p in zip(caches, pools):
                B.release_pages(c, p, i32(seqs))
            continue
        q, k, v = rows(i, counts, hkv, g, d)
        c, pool, ids = caches[0], pools[0], i32(seqs)
        plan = B.alloc_plan(slots, sum(counts))
        B.plan_pages(c, pool, i32(counts), plan, seq_ids=ids, max_count=most)
        batch = plan.batch(most, ids)
        B.append_q8(c, k, v, batch)
        before = w.clone()
        if diff:
            o = B.attend_diff_q8(c, q, lam, batch, gain=gain, **score)
            check_diff(c, q, counts, o, lam, gain, seq_ids=seqs, **score)
        else:
            o = B.attend_q8(c, q, batch, alpha=alpha, **score)
            check_attend(c, q, counts, o, seq_ids=seqs, alpha=alpha, **score)
        B.weigh_q8(c, w, q, o.tau, batch, alpha=alpha, decay=decay, **score)
        check_weights(c, q, counts, o.tau, before, w, alpha, decay=decay, seq_ids=seqs, **score)
        held = state(c, pool, w)
        busy = [s for s, n in zip(seqs, counts) if n]
        want = expect(c, held, code, busy, keep, above, sinks, recent)
        B.evict_q8(c, pool, w, ids, keep, above=above, sinks=sinks, recent=recent, count=plan.count)
        got = state(c, pool, w)
        for name in ("lens", "count", "free", "ks", "vs", "w"):
            assert same(got[name], want[name]), (i, name)
        os_ = step.run(i32(counts), ids, q, k, v)
        torch.cuda.synchronize()
        n = sum(counts)
        assert torch.equal(o.out, os_.out[:n]) and torch.equal(torch.nan_to_num(o.tau), torch.nan_to_num(os_.tau[:n]))
        there = state(caches[1], pools[1], step.budget.weights)
        assert all(torch.equal(got[name], there[name]) for name in got), i
    assert max(caches[0].seq_lens.tolist()) <= above
    assert caches[0].device_status() == 0 and caches[1].device_status() == 0


def test_a_prompt_by_its_last_rows_then_single_tokens():
    """A long prompt is appended in one piece, weighed by its last 32 rows alone and shortened, and decoded on: what
    is kept attends as the shortened sequence does."""
    hkv, g, d, P = 2, 4, 128, 32
    c, pool = B.QuantCache(hkv, g, d, P, 1, 80, 80, torch.int8), B.PagePool.full(80)
    q, k, v = rows(1, [2000], hkv, g, d)
    ids, w = i32([0]), B.alloc_weights(c)
    plan = B.alloc_plan(1, 2000)
    B.plan_pages(c, pool, i32([2000]), plan)
    B.append_q8(c, k, v, plan.batch(2000))
    last = B.Batch(i32([0]), i32([32]), 32, 32)
    tau = B.attend_q8(c, q[-32:], last).tau
    before = torch.full_like(w, float("nan"))   # nothing of it may be read
    w.copy_(before)
    B.weigh_q8(c, w, q[-32:], tau, last, fresh=i32([2000]))
    check_weights(c, q[-32:], [32], tau, before, w, fresh=[2000])
    B.evict_q8(c, pool, w, ids, 500, sinks=4, recent=100)
    assert c.seq_lens.tolist() == [500] and int(pool.free_count) == 80 - 16
    for i in range(3):
        q, k, v = rows(2 + i, [1], hkv, g, d)
        B.plan_pages(c, pool, i32([1]), plan := B.alloc_plan(1, 1))
        B.append_q8(c, k, v, plan.batch(1))
        check_attend(c, q, [1], B.attend_q8(c, q, plan.batch(1)))
    assert c.device_status() == 0 and c.seq_lens.tolist() == [503]


def test_steps_given_one_budget_keep_weights_of_their_own():
    hkv, g, d, P = 2, 4, 64, 16
    budget = B.KeyBudget(20, 24, 2, 6)
    q, k, v = rows(3, [1], hkv, g, d)
    caches = [B.QuantCache(hkv, g, d, P, 1, 4, 4, torch.int8) for _ in range(2)]
    steps = [B.QuantStep(c, B.PagePool.full(4), 1, budget=budget) for c in caches]
    assert budget.weights is None
    steps[0].run(i32([1]), i32([0]), q, k, v)
    assert float(steps[0].budget.weights.sum()) > 0 and not steps[1].budget.weights.any()
