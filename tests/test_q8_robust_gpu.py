"""The 8-bit cache where it is used in ways that single calls in an empty
device do not show: clusters that start one by one, calls on other streams,
non-finite queries, long and dense supports, steps that ask for too much."""

import numpy as np
import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

from q8_cases import batch_of, check_attend, dense, empty_cache, filled, i32

pytestmark = pytest.mark.gpu


def test_entmax_clusters_that_start_beside_other_work_give_the_same_bits():
    """Blocks of a cluster find their multiprocessors taken by another stream's products."""
    c, q = filled("int8", [9000], [1], hkv=4, g=4)
    batch = batch_of([1])
    first = B.attend_q8(c, q, batch, alpha=1.5)
    ws, o = B.alloc_attend_workspace(c, batch, 1.5), B.alloc_attend_outputs(c, batch)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x = torch.randn(2048, 2048, device="cuda").bfloat16()
    torch.cuda.synchronize()
    for _ in range(40):
        with torch.cuda.stream(side):
            for _ in range(4):
                x @ x
        B.attend_q8(c, q, batch, alpha=1.5, workspace=ws, outputs=o)
        torch.cuda.current_stream().synchronize()
        assert torch.equal(o.out, first.out) and torch.equal(o.tau, first.tau)
    torch.cuda.synchronize()
    assert c.device_status() == 0


ORDERS = [float(np.float32(a)) for a in (1.002, 1.1, 1.25, 1.5, 1.75, 2.0, 2.2, 2.5, 3.0, 4.0, 6.0)]


def _sum_tol(alpha):
    """Of an output Σ p·v, v 0 or 1: its rounding to bf16 (half a step, 2^-8 of up to 1), each weight's to a half
    (2^-11), the sum's own bound 2^-14 + β·2^-21, the weights' powers (β·2^-21 again: the solve's and the weights'
    may differ) and 127 · fl32(1/127) for a 1 (2^-24)."""
    return 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -20 / (alpha - 1.0) + 2.0 ** -24


@pytest.mark.parametrize("alpha", ORDERS)
@pytest.mark.parametrize("n", [1, 33, 1000, 10000, 100001])
def test_weights_of_equal_keys_add_up_to_one(alpha, n):
    """Scores that are exactly equal, V all ones: the output is the weights' sum, with and without the scores
    handed round a cluster (1000 and 10000 keys)."""
    c = empty_cache("int8", [n, 3], hkv=2, g=4, d=64, P=16)
    x = torch.ones(n + 3, 2, 64, device="cuda").bfloat16()
    B.append_q8(c, x, x, batch_of([n, 3]))
    gen = torch.Generator(device="cuda").manual_seed(n)
    q = torch.randn(2, 8, 64, generator=gen, device="cuda").bfloat16()
    o = B.attend_q8(c, q, batch_of([1, 1]), alpha=alpha)
    assert c.device_status() == 0
    assert float((o.out.float() - 1.0).abs().max()) <= _sum_tol(alpha)
    # τ = z − n^{1−α}; a score is good to 2^-20·(Σ|q||k|/√d + 1), and τ is rounded to fp32
    z = (alpha - 1.0) * q.double().sum(-1) / 8.0
    want = z - torch.tensor([n, 3], device="cuda").double()[:, None] ** (1.0 - alpha)
    tol = 2.0 ** -20 * (alpha - 1.0) * (q.double().abs().sum(-1) / 8.0 + 1.0) + 2.0 ** -23 * want.abs()
    # and by what the sum's bound lets it move: |S − 1|·(z − τ)/β
    tol += (alpha - 1.0) * (2.0 ** -14 + 2.0 ** -21 / (alpha - 1.0)) * (z - want)
    assert bool(((o.tau.double() - want).abs() <= tol).all())


def _share(D, m, alpha):
    """Of one key whose z lies D above those of m equal ones: the m keys' share of the weight, in 64 bits:
    m·ρ^β + (D + ρ)^β = 1 by bisection on log2 ρ."""
    beta, lo, hi = 1.0 / (alpha - 1.0), -400.0, 0.0
    for _ in range(200):
        mid = 0.5 * (lo + hi)
        lo, hi = (lo, mid) if m * 2.0 ** (mid * beta) + (D + 2.0 ** mid) ** beta >= 1.0 else (mid, hi)
    return m * 2.0 ** (hi * beta)


@pytest.mark.parametrize("alpha", ORDERS[2:-1])
@pytest.mark.parametrize("m", [40, 1000, 100000])
@pytest.mark.parametrize("D", [0.9, 0.3, 1e-3])
def test_one_key_above_many_equal_ones(alpha, m, D):
    """The threshold lies next to the many keys' score, above order 2 far nearer than a float's step at D."""
    d, P = 64, 16
    c = empty_cache("int8", [m + 1], hkv=1, g=2, d=d, P=P)
    k, v = torch.ones(m + 1, 1, d, device="cuda"), torch.ones(m + 1, 1, d, device="cuda")
    k[P:] = 0.5   # the strong key's page holds equal keys of its own too: they are masked below
    v[:P] = 0.0
    B.append_q8(c, k.bfloat16(), v.bfloat16(), batch_of([m + 1]))
    K = dense(c, 0, 0, "k")
    diff = float((K[P - 1] - K[P])[0])
    q = torch.zeros(1, 2, d, device="cuda")
    q[0, 0, 0] = q[0, 1, 0] = 1.0
    scale = D / ((alpha - 1.0) * diff)
    o = B.attend_q8(c, q.bfloat16(), batch_of([1]), alpha=alpha, scale=scale,
                    first_key=torch.tensor([P - 1], dtype=torch.int32, device="cuda"))
    assert c.device_status() == 0
    many = m + 1 - P
    share = _share(D, many, alpha)
    # V is 1 for the many keys and 0 for the strong one. D is good to 2^-20: the scores' common factor has four
    # roundings of 2^-24, each score (2D and D) two of its own, the difference one. The share at both ends:
    ends = [_share(D * (1 + s * 2.0 ** -20), many, alpha) for s in (-1, 1)]
    tol = _sum_tol(alpha) + max(abs(e - share) for e in ends)
    got = float(o.out[0, 0, 0])
    assert abs(got - share) <= tol, (got, share, tol)
    assert torch.equal(o.out[0, 0], o.out[0, 1])


@pytest.mark.parametrize("alpha", [1.25, 1.5, 2.0, 3.0])
def test_dense_supports_add_up_to_one(alpha):
    """Random scores close together: most of 60000 keys in the support, V all ones."""
    n = 60000
    c = empty_cache("e4m3", [n], hkv=2, g=4, d=64, P=32)
    gen = torch.Generator(device="cuda").manual_seed(5)
    k = torch.randn(n, 2, 64, generator=gen, device="cuda").bfloat16()
    B.append_q8(c, k, torch.ones_like(k), batch_of([n]))
    q = torch.randn(1, 8, 64, generator=gen, device="cuda").bfloat16()
    for scale in (1e-7, 1e-4, 1e-2, 0.1):
        o = B.attend_q8(c, q, batch_of([1]), alpha=alpha, scale=scale)
        assert c.device_status() == 0
        assert float((o.out.float() - 1.0).abs().max()) <= _sum_tol(alpha), scale


@pytest.mark.parametrize("alpha,counts", [(1.0, [1, 1, 1]), (1.25, [1, 1, 1]), (1.5, [1, 1, 1]), (2.0, [1, 1, 1]),
                                          (3.0, [1, 1, 1]), (1.0, [3, 2, 1]), (1.0, [3, 2, 9]), (1.0, [120, 70, 1])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_a_non_finite_query_gives_nan_in_its_own_row_and_head(alpha, counts, bad, code):
    """Sequences of many tokens and of one (where an infinity's score can be -inf, a masked key's), rows that see
    nothing beside them; every other row and head keeps its bits."""
    lens = [500, 90, counts[2]]
    c, q = filled(code, lens, counts, hkv=2, g=3, d=64, P=16)
    batch = batch_of(counts)
    fk = torch.zeros(sum(counts), dtype=torch.int32, device="cuda")
    fk[1 if counts[0] > 1 else 0] = 10 ** 6  # sees no key
    clean = B.attend_q8(c, q, batch, alpha=alpha, first_key=fk)
    q2, spoilt = q.clone(), torch.zeros(sum(counts), 6, dtype=torch.bool, device="cuda")
    blind = fk > 0
    for row, head, i in ((0, 1, 3), (counts[0], 4, 0), (counts[0], 0, 63), (sum(counts) - 1, 2, 17),
                         (sum(counts) - 1, 3, 18), (int(blind.nonzero()[0]), 5, 9)):
        q2[row, head, i] = bad
        spoilt[row, head] = not blind[row]
    o = B.attend_q8(c, q2, batch, alpha=alpha, first_key=fk)
    assert c.device_status() == 0
    assert bool(torch.isnan(o.out[spoilt]).all()) and bool(torch.isnan(o.tau[spoilt]).all())
    assert torch.equal(o.out[~spoilt], clean.out[~spoilt])
    assert torch.equal(o.tau[~spoilt].nan_to_num(7.0), clean.tau[~spoilt].nan_to_num(7.0))
    assert not o.out[blind].any() and bool(torch.isnan(o.tau[blind]).all())


def test_entmax_scores_past_the_largest_float_give_nan():
    c, q = filled("int8", [200], [1], hkv=1, g=2, d=64, P=16)
    q2 = q.clone()
    q2[0, 0] = 2.0 ** 120
    o = B.attend_q8(c, q2, batch_of([1]), alpha=1.5, scale=2.0 ** 20)
    base = B.attend_q8(c, q, batch_of([1]), alpha=1.5, scale=2.0 ** 20)
    assert bool(torch.isnan(o.out[0, 0]).all()) and bool(torch.isnan(o.tau[0, 0]))
    assert torch.equal(o.out[0, 1], base.out[0, 1]) and c.device_status() == 0


@pytest.mark.parametrize("alpha,counts", [(1.0, [1, 1]), (1.5, [1, 1]), (1.0, [90, 40])])
def test_calls_on_a_side_stream_make_their_own_buffers_there(alpha, counts):
    """The current stream is kept busy before each call and takes what the call dropped after it: the outputs
    neither lose to a late fill nor to another tensor in the workspace's place."""
    c, q = filled("int8", [4000, 900], counts, hkv=4, g=4)
    batch = batch_of(counts)
    want = B.attend_q8(c, q, batch, alpha=alpha)
    first = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    rows = B.read_q8(c, first, batch)
    size = B.attend_workspace_bytes(c, batch, alpha)
    x = torch.randn(4096, 4096, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for _ in range(10):
            x @ x  # (a few ms)
        o = B.attend_q8(c, q, batch, alpha=alpha, stream=side)
        k, v = B.read_q8(c, first, batch, stream=side)
        torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xff)
        torch.cuda.synchronize()
        assert torch.equal(o.out, want.out) and torch.equal(o.tau, want.tau)
        assert torch.equal(k, rows[0]) and torch.equal(v, rows[1])
    assert c.device_status() == 0


def test_decode_on_a_side_stream_makes_its_own_buffers_there():
    cache = B.PagedCache(2, 4, 128, 16, 1, 40, 40, torch.bfloat16)
    cache.block_table[0] = torch.arange(40, device="cuda")
    kv = torch.randn(2, 1, 2, 600, 128, device="cuda").bfloat16()
    B.append(cache, kv[0], kv[1])
    q = torch.randn(1, 8, 128, device="cuda").bfloat16()
    want = B.decode(cache, q, 1.5, "full")
    x = torch.randn(4096, 4096, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        x @ x
    o = B.decode(cache, q, 1.5, "full", stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o.page_ids, want.page_ids) and torch.equal(o.n_sel, want.n_sel)
    torch.testing.assert_close(o.out, want.out, rtol=1e-5, atol=1e-5)  # (its sums' order is not fixed)


@pytest.mark.parametrize("most,alpha,news", [(1, 1.5, [2, 0, 0, 0]), (1, 1.0, [0, 0, 3, 1]), (40, 1.0, [41, 0, 7, 0]),
                                             (3, 1.0, [1, 4, 0, 2])])
def test_a_step_refuses_a_slot_over_its_bound_and_leaves_its_sequence(most, alpha, news):
    c = B.QuantCache(2, 4, 64, 16, 6, 20, 60, torch.int8)
    pool = B.PagePool.full(60)
    step = B.QuantStep(c, pool, 4, most, alpha=alpha)
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = [3, 1, 0, 5]

    def run(counts):
        n = min(sum(counts), 4 * most)
        qkv = torch.randn(n, 12, 64, generator=gen, device="cuda").bfloat16()
        return qkv[:, :8], step.run(i32(counts), i32(ids), qkv[:, :8], qkv[:, 8:10], qkv[:, 10:])

    run([most] * 4)
    lens, table, free = c.seq_lens.tolist(), c.block_table.clone(), pool.free_count.item()
    codes = c.k_pool.clone()
    assert c.device_status() == 0
    q, o = run(news)
    assert c.device_status() == B.DEV_BAD_BATCH
    c.status.zero_()
    fine = [n if n <= most else 0 for n in news]
    for b, n in zip(ids, fine):
        lens[b] += n
    assert c.seq_lens.tolist() == lens and step.plan.count.tolist() == fine
    used = sum(-(-x // 16) for x in lens)
    assert pool.free_count.item() == 60 - used and free >= pool.free_count.item()
    over = [b for b, n in zip(ids, news) if n > most]
    assert torch.equal(c.block_table[over], table[over])
    for b in over:
        held = table[b, :-(-lens[b] // 16)].long()
        assert torch.equal(c.k_pool[held], codes[held])
    check_attend(c, q, fine, o, seq_ids=ids, alpha=alpha, start=step.plan.start.tolist())
    q, o = run([1, 1, 1, 1])  # and the next step sees what was written alone
    assert c.device_status() == 0
    check_attend(c, q, [1] * 4, o, seq_ids=ids, alpha=alpha)


def test_a_step_takes_rows_of_its_own_shapes_only():
    """copy_ would repeat one row, head or value for all: refused before anything changes."""
    c = B.QuantCache(2, 4, 64, 16, 3, 8, 20, torch.int8)
    step = B.QuantStep(c, B.PagePool.full(20), 3, 2)
    n, ids = i32([2, 1, 0]), i32([0, 1, 2])
    r = lambda rows, heads, d=64: torch.randn(rows, heads, d, device="cuda").bfloat16()  # noqa: E731
    q, k, v = r(3, 8), r(3, 2), r(3, 2)
    for bad in ((n, ids, q, k[:1], v), (n, ids, q, k, v[0]), (n, ids, q[:, :1], k, v),
                (n, ids, r(7, 8), r(7, 2), r(7, 2)), (n[:1], ids, q, k, v), (n, ids[:1], q, k, v),
                (n, ids, q, r(3, 2, 1), v)):
        with pytest.raises(B.EntmaxKVError):
            step.run(*bad)
    torch.cuda.synchronize()
    assert c.seq_lens.tolist() == [0, 0, 0] and not step.k.any()
    step.run(n, ids, q, k, v)
    assert c.seq_lens.tolist() == [2, 1, 0] and torch.equal(step.k[:3], k)


def test_planning_with_a_bound_and_without():
    def state():
        t = B.PageTable(i32([[-1] * 8] * 3), i32([0, 5, 0]), 16, 20)
        t.block_table[1, 0] = 19
        return t, B.PagePool(torch.arange(19, dtype=torch.int32, device="cuda"), i32([19])), B.alloc_plan(3, 60)

    t, pool, plan = state()
    pool = B.PagePool(torch.cat([pool.free_pages, i32([0])]), pool.free_count)
    B.plan_pages(t, pool, i32([17, 30, 4]), plan, max_count=17)
    assert plan.start.tolist() == [0, 17, 47] and plan.count.tolist() == [17, 0, 4]
    assert t.seq_lens.tolist() == [17, 5, 4] and pool.free_count.item() == 16
    assert t.block_table[1].tolist() == [19] + [-1] * 7 and t.device_status() == B.DEV_BAD_BATCH
    assert plan.positions.tolist() == list(range(17)) + [-1] * 30 + [0, 1, 2, 3] + [-1] * 9
    t, pool, plan = state()
    pool = B.PagePool(torch.cat([pool.free_pages, i32([0])]), pool.free_count)
    B.plan_pages(t, pool, i32([17, 30, 4]), plan)
    assert plan.count.tolist() == [17, 30, 4] and t.device_status() == 0
