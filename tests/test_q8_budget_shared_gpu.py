"""Several steps over one cache share the weights of its keys: prompts in pieces by one captured step, single tokens by
another, and weights that the caller added, against the same calls one by one with one tensor."""

import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

from q8_cases import DT, i32
from test_q8_budget_gpu import rows
from test_q8_evict_gpu import state

pytestmark = pytest.mark.gpu


def eager(c, pool, w, most, counts, seqs, q, k, v, b, decay):
    ids, plan = i32(seqs), B.alloc_plan(len(seqs), sum(counts))
    B.plan_pages(c, pool, i32(counts), plan, seq_ids=ids, max_count=most)
    batch = plan.batch(most, ids)
    B.append_q8(c, k, v, batch)
    o = B.attend_q8(c, q, batch)
    B.weigh_q8(c, w, q, o.tau, batch, decay=decay)
    B.evict_q8(c, pool, w, ids, b.keep, above=b.above, sinks=b.sinks, recent=b.recent, count=plan.count)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("given", [False, True])
def test_a_step_of_prompts_and_one_of_tokens(code, given):
    """Prompts of 30 tokens a piece and single tokens behind them, sequences that leave, and others that get their
    pages: after every step the tokens' step knows what the prompts' step weighed and moved."""
    hkv, g, d, P, pages = 2, 4, 64, 16, 30
    caches = [B.QuantCache(hkv, g, d, P, 4, 12, pages, DT[code]) for _ in range(2)]
    pools = [B.PagePool.full(pages) for _ in range(2)]
    w = B.alloc_weights(caches[0])
    mine = B.alloc_weights(caches[1]) if given else None
    budget = B.KeyBudget(48, 56, 2, 10, decay=0.9, weights=mine)
    steps = {most: B.QuantStep(caches[1], pools[1], 2, most, budget=budget) for most in (30, 1)}
    assert steps[1].budget.weights is steps[30].budget.weights is (mine if given else caches[1].key_weights())
    runs = [(30, [30, 17], [0, 1]), (30, [30, 30], [0, 1]), (30, [5, 30], [0, 1])] + [(1, [1, 1], [0, 1])] * 12
    runs += [("release", [0]), (30, [30, 1], [2, 1]), (30, [30, 0], [2, 1])] + [(1, [1, 1], [2, 1])] * 12
    for i, run in enumerate(runs):
        if run[0] == "release":
            for c, p in zip(caches, pools):
                B.release_pages(c, p, i32(run[1]))
            continue
        most, counts, seqs = run
        q, k, v = rows(100 + i, counts, hkv, g, d)
        eager(caches[0], pools[0], w, most, counts, seqs, q, k, v, budget, 0.9)
        steps[most].run(i32(counts), i32(seqs), q, k, v)
        torch.cuda.synchronize()
        a, b = state(caches[0], pools[0], w), state(caches[1], pools[1], steps[most].budget.weights)
        assert all(torch.equal(a[name], b[name]) for name in a), i
    assert all(c.device_status() == 0 for c in caches) and int(caches[1].seq_lens.max()) <= 56


def test_what_the_caller_weighs_is_the_steps_too():
    """A prompt appended and weighed by calls, then shortened by a step of single tokens: its heavy keys stay."""
    hkv, g, d, P = 1, 2, 64, 16
    c, pool = B.QuantCache(hkv, g, d, P, 1, 12, 12, torch.int8), B.PagePool.full(12)
    step = B.QuantStep(c, pool, 1, budget=B.KeyBudget(40, sinks=0, recent=4))
    q, k, v = rows(1, [100], hkv, g, d)
    plan = B.plan_pages(c, pool, i32([100]), B.alloc_plan(1, 100))
    batch = plan.batch(100)
    B.append_q8(c, k, v, batch)
    w = c.key_weights()
    assert w is step.budget.weights and c.key_weights() is w
    B.weigh_q8(c, w, q, B.attend_q8(c, q, batch).tau, batch)
    before = w[c.block_table[0, :7].long(), 0].reshape(-1)[:100].clone()
    q, k, v = rows(2, [1], hkv, g, d)
    step.run(i32([1]), i32([0]), q, k, v)
    torch.cuda.synchronize()
    assert c.seq_lens.tolist() == [40]
    after = w[c.block_table[0, :3].long(), 0].reshape(-1)[:40]
    # of the first 97 keys the 36 heaviest stay, and weights only grew: none is below the 36th of before
    heavy = before[:97].sort(descending=True).values[35]
    assert float(after[:36].min()) >= float(heavy) > 0.0


def test_caches_keep_weights_of_their_own():
    caches = [B.QuantCache(2, 4, 64, 16, 1, 4, 4, torch.int8) for _ in range(2)]
    a, b = (c.key_weights() for c in caches)
    assert a is not b and a.data_ptr() != b.data_ptr() and a.shape == (4, 2, 16) and not bool(a.any())


def test_the_tensor_is_not_made_inside_a_capture():
    """(There each replay would clear it.)"""
    c = B.QuantCache(2, 4, 64, 16, 1, 4, 4, torch.int8)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        with pytest.raises(B.EntmaxKVError, match="capture"):
            c.key_weights()
    w = c.key_weights()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        assert c.key_weights() is w
