"""A serving run over the 8-bit cache: plan, append, attend, release, eagerly
and as the captured step, against one another and the oracle."""

import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

from q8_cases import DT, check_attend, i32

pytestmark = pytest.mark.gpu


def _step_inputs(seed, counts, hkv, g, d):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(sum(counts), (g + 2) * hkv, d, generator=gen, device="cuda").bfloat16()
    return qkv[:, :g * hkv], qkv[:, g * hkv:g * hkv + hkv], qkv[:, g * hkv + hkv:]


@pytest.mark.parametrize("code,most,alpha", [("int8", 1, 1.0), ("e4m3", 1, 1.5), ("int8", 40, 1.0), ("e4m3", 3, 1.0)])
def test_captured_step_matches_eager_calls_and_the_oracle(code, most, alpha):
    hkv, g, d, P, slots, rows = 2, 4, 128, 16, 4, 6
    caches = [B.QuantCache(hkv, g, d, P, rows, 30, 64, DT[code]) for _ in range(2)]
    pools = [B.PagePool.full(64) for _ in range(2)]
    score = dict(softcap=12.0, window=60)
    step = B.QuantStep(caches[1], pools[1], slots, most, alpha=alpha, **score)
    # prompts, decodes with an idle slot, a sequence that leaves and one that takes its row
    runs = [([most] * 4, [0, 1, 2, 3]), ([1, min(2, most), 0, most], [0, 1, 99, 3]), ([1, 1, 1, 1], [3, 2, 1, 0]),
            ("release", [1]), ([most, 1, 1, 0], [1, 5, 0, 0]), ([1, 1, 1, 1], [1, 5, 0, 3])]
    for i, (counts, seqs) in enumerate(runs):
        if counts == "release":
            for c, p in zip(caches, pools):
                B.release_pages(c, p, i32(seqs))
            continue
        q, k, v = _step_inputs(i, counts, hkv, g, d)
        c, pool = caches[0], pools[0]
        plan = B.alloc_plan(slots, sum(counts))
        B.plan_pages(c, pool, i32(counts), plan, seq_ids=i32(seqs))
        batch = plan.batch(most, i32(seqs))
        B.append_q8(c, k, v, batch)
        o = B.attend_q8(c, q, batch, alpha=alpha, **score)
        os_ = step.run(i32(counts), i32(seqs), q, k, v)
        torch.cuda.synchronize()
        n = sum(counts)
        assert torch.equal(o.out, os_.out[:n]) and torch.equal(o.tau, os_.tau[:n])
        assert torch.equal(plan.positions, step.plan.positions[:n]) and torch.equal(plan.slots, step.plan.slots[:n])
        check_attend(c, q, counts, o, seq_ids=seqs, alpha=alpha, **score)
    a, b = caches
    assert torch.equal(a.k_pool.view(torch.int8), b.k_pool.view(torch.int8)) and torch.equal(a.v_scale, b.v_scale)
    assert torch.equal(a.seq_lens, b.seq_lens) and torch.equal(pools[0].free_count, pools[1].free_count)
    assert a.device_status() == 0 and b.device_status() == 0


def test_a_full_pool_refuses_a_slot_and_the_rest_goes_on():
    c = B.QuantCache(1, 2, 64, 16, 3, 8, 4, torch.int8)
    pool = B.PagePool.full(4)
    counts, seqs = [40, 30, 1], [0, 1, 2]
    q, k, v = _step_inputs(0, counts, 1, 2, 64)
    plan = B.alloc_plan(3, 71)
    B.plan_pages(c, pool, i32(counts), plan)
    assert plan.count.tolist() == [40, 0, 0] and c.device_status() == B.DEV_CAPACITY
    batch = plan.batch(40)
    o = B.alloc_attend_outputs(c, batch)
    o.out.fill_(5.0)
    B.append_q8(c, k, v, batch)
    B.attend_q8(c, q, batch, outputs=o)
    assert bool((o.out[40:] == 5.0).all()) and c.seq_lens.tolist() == [40, 0, 0]
    check_attend(c, q, [40, 0, 0], o, seq_ids=seqs, start=[0, 40, 70])


def test_two_captured_steps_do_not_share_a_workspace():
    """Graphs of two steps over one cache, replayed on two streams at once, give what they give alone."""
    hkv, g, d = 2, 4, 64
    made = []
    for s in range(2):
        c = B.QuantCache(hkv, g, d, 16, 2, 200, 400, torch.int8)
        pool = B.PagePool.full(400)
        plan = B.alloc_plan(2, 3000)
        B.plan_pages(c, pool, i32([1700, 1300]), plan)
        gen = torch.Generator(device="cuda").manual_seed(s)
        kv = torch.randn(2, 3000, hkv, d, generator=gen, device="cuda").bfloat16()
        B.append_q8(c, kv[0], kv[1], plan.batch(1700))
        made.append((c, B.QuantStep(c, pool, 2), *_step_inputs(50 + s, [1, 1], hkv, g, d)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for r in range(5):
        for (c, step, q, k, v), st in zip(made, streams):
            with torch.cuda.stream(st):
                step.run(i32([1, 1]), i32([0, 1]), q, k, v)
        torch.cuda.synchronize()
        for c, step, q, k, v in made:
            check_attend(c, q, [1, 1], step.outputs, seq_ids=[0, 1])
