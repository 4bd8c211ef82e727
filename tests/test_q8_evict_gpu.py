"""Eviction from the 8-bit cache, bit for bit against the oracle."""

import numpy as np
import pytest
import torch

from oracle import q8 as oq
from sparse_entmax_attention_gb300 import binding as B

from q8_cases import filled, i32

pytestmark = pytest.mark.gpu


def make(code, lens, hkv=2, d=128, P=32, seed=0, spare=9):
    c, _ = filled(code, lens, [1] * len(lens), hkv=hkv, g=2, d=d, P=P, seed=seed, spare=spare)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    # pages of unlike loudness
    for s in (c.k_scale, c.v_scale):
        s.mul_(torch.exp(0.5 * torch.randn(s.shape, generator=gen, device="cuda")))
    used = torch.zeros(c.cfg.num_phys_pages, dtype=torch.bool)
    for b, n in enumerate(lens):
        used[c.block_table[b, :-(-n // P)].long().cpu()] = True
    free = torch.nonzero(~used).flatten().int().cuda()
    stack = torch.full((c.cfg.num_phys_pages,), -7, dtype=torch.int32, device="cuda")
    stack[:len(free)] = free
    return c, B.PagePool(stack, i32([len(free)]))


def spread_weights(c, seed=0, ties=0.3):
    gen = torch.Generator(device="cuda").manual_seed(seed + 50)
    w = torch.exp(2.0 * torch.randn(B.alloc_weights(c).shape, generator=gen, device="cuda"))
    w[torch.rand(w.shape, generator=gen, device="cuda") < ties] = 0.0
    return w


def state(c, pool, w):
    codes = [p.view(torch.int8).clone() for p in (c.k_pool, c.v_pool)]
    return dict(k=codes[0], v=codes[1], ks=c.k_scale.clone(), vs=c.v_scale.clone(), lens=c.seq_lens.clone(),
                free=pool.free_pages.clone(), count=pool.free_count.clone(), w=None if w is None else w.clone(),
                table=c.block_table.clone())


def expect(c, s, code, seqs, keep, above, sinks, recent):
    """The state after eviction, from the one before."""
    P, hkv, d = c.cfg.page_size, c.cfg.num_kv_heads, c.cfg.head_dim
    table, out = s["table"].cpu().numpy(), {k: None if v is None else v.cpu().clone() for k, v in s.items()}
    count = int(s["count"])
    for seq in seqs:
        L = int(out["lens"][seq])
        if L <= above:
            continue
        ph = table[seq, :-(-L // P)]
        for h in range(hkv):
            w = np.zeros(L) if s["w"] is None else s["w"][ph, h].reshape(-1)[:L].double().cpu().numpy()
            kept = oq.kept_keys(w, keep, sinks, recent)
            for side in "kv":
                held = s[side][ph, h].reshape(-1, d)[:L]
                scales = np.repeat(s[side + "s"][ph, h].cpu().numpy(), P)[:L]
                vals = held.cpu().view(torch.int8 if code == "int8" else torch.float8_e4m3fn).double().numpy()
                rows, now = oq.evict_rows(vals, scales, kept, P, code)
                for p in range(len(now)):
                    part = torch.from_numpy(rows[p * P:p * P + P])
                    part = part.to(torch.int8) if code == "int8" else part.float().to(torch.float8_e4m3fn).view(torch.int8)
                    out[side][ph[p], h, :len(part)] = part
                    out[side + "s"][ph[p], h] = now[p]
            if s["w"] is not None:
                for i, j in enumerate(kept):
                    out["w"][ph[i // P], h, i % P] = s["w"][ph[j // P], h, j % P].cpu()
        for p in range(len(ph) - 1, -(-keep // P) - 1, -1):
            out["free"][count] = int(ph[p])
            count += 1
        out["lens"][seq] = keep
    out["count"][0] = count
    return out


def same(a, b):
    return torch.equal(torch.nan_to_num(a.float().cpu(), nan=1e33), torch.nan_to_num(b.float().cpu(), nan=1e33))


def check(c, pool, w, code, seqs, keep, above=0, sinks=0, recent=0, status=0, refused=()):
    before = state(c, pool, w)
    want = expect(c, before, code, [s for s in seqs if s not in refused], keep, above or keep, sinks, recent)
    B.evict_q8(c, pool, w, i32(seqs), keep, above=above, sinks=sinks, recent=recent)
    torch.cuda.synchronize()
    assert c.device_status() == status
    got = state(c, pool, w)
    for k in ("lens", "count", "free", "ks", "vs", "k", "v", "w", "table"):
        if want[k] is not None:
            if k in "kv":  # (−0 is 0 in e4m3)
                t = torch.int8 if code == "int8" else torch.float8_e4m3fn
                assert same(got[k].view(t), want[k].view(t)), k
            else:
                assert same(got[k], want[k]), k


@pytest.mark.parametrize("code,d,P", [("int8", 128, 32), ("e4m3", 128, 16), ("int8", 64, 16), ("e4m3", 64, 32)])
@pytest.mark.parametrize("keep,sinks,recent", [(64, 0, 0), (70, 4, 20), (1, 0, 0), (33, 33, 0), (100, 0, 100), (129, 1, 1)])
def test_lengths_around_the_limit(code, d, P, keep, sinks, recent):
    lens = [1, keep - 1 or 1, keep, keep + 1, keep + P, 5 * keep + 3, 700]
    c, pool = make(code, lens, d=d, P=P, seed=keep)
    check(c, pool, spread_weights(c), code, [3, 0, 6, 2, 5, 1, 4], keep, sinks=sinks, recent=recent)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("n,keep,P", [(9000, 8999, 32), (9000, 5000, 16), (20000, 100, 32), (40000, 9000, 16)])
def test_long_sequences_over_several_waves(code, n, keep, P):
    """More pages than the warps of a cluster hold at once, both for the keys that stay and those looked at."""
    c, pool = make(code, [n, 50], hkv=1, d=64, P=P, seed=1)
    check(c, pool, spread_weights(c), code, [0, 1], keep, sinks=3, recent=64)


def test_more_keys_than_shared_memory_holds():
    n = 8 * 16384 + 5000
    c, pool = make("int8", [n], hkv=1, d=64, P=32, seed=1)
    check(c, pool, spread_weights(c), "int8", [0], 4000, sinks=3, recent=64)


@pytest.mark.parametrize("ties", ["zero", "one", "signs", "odd"])
def test_equal_and_odd_weights(ties):
    c, pool = make("int8", [700, 333], seed=2, P=16, d=64)
    w = torch.zeros_like(B.alloc_weights(c))
    if ties == "one":
        w += 1.0
    if ties == "signs":
        w[:, :, ::2] = -0.0
        w[:, :, 1::5] = -1.0
    if ties == "odd":
        w = spread_weights(c)
        w[:, :, 3], w[:, :, 5], w[:, :, 7], w[:, :, 9] = float("nan"), float("inf"), -float("inf"), 1e-42
    check(c, pool, w, "int8", [0, 1], 100, sinks=2, recent=5)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_pages_whose_scale_is_zero(code):
    """All of a sequence's pages, every second one, and pages of the smallest scale that append writes."""
    c, pool = make(code, [700, 650, 333], seed=4, P=16, d=64)
    for s in (c.k_scale, c.v_scale):
        s[c.block_table[0, :44].long()] = 0.0
        s[c.block_table[1, :41:2].long()] = 0.0
        s[c.block_table[2, :21].long()] = 2.0 ** -96
    check(c, pool, spread_weights(c), code, [0, 1, 2], 100, sinks=2, recent=5)


def test_above_leaves_sequences_until_they_pass_it():
    c, pool = make("e4m3", [100, 130, 131, 400], P=16)
    check(c, pool, spread_weights(c), "e4m3", [0, 1, 2, 3], 90, above=130)


def test_without_weights_the_ends_stay():
    c, pool = make("int8", [300, 64], P=32)
    check(c, pool, None, "int8", [0, 1], 64, sinks=10, recent=54)


def test_again_and_again():
    """A sequence that is shortened, shortened again and shortened on: from the state that it left."""
    c, pool = make("e4m3", [900], P=16, d=64)
    w = spread_weights(c)
    for keep in (700, 699, 300, 300, 17):
        check(c, pool, w, "e4m3", [0], keep, sinks=2, recent=3)


def test_refused_slots_are_left_as_they_were():
    c, pool = make("int8", [300, 300, 300, 300], P=32)
    c.block_table[2, 7] = c.cfg.num_phys_pages
    w = spread_weights(c)
    check(c, pool, w, "int8", [0, 99, 2, 3, 0, -1], 50, status=B.DEV_BAD_SEQ_ID | B.DEV_BAD_PAGE_TABLE | B.DEV_BAD_BATCH,
          refused=(99, 2, -1))
    assert c.seq_lens.tolist() == [50, 300, 300, 50]


def test_outputs_of_their_own_leave_the_inputs():
    c, pool = make("int8", [300, 40, 500], P=32, seed=5)
    w = spread_weights(c)
    before = state(c, pool, w)
    want = expect(c, before, "int8", [2, 1], 64, 64, 1, 8)
    lens, count, w_out = torch.full_like(c.seq_lens, -3), i32([-3]), torch.full_like(w, -3.0)
    B.evict_q8(c, pool, w, i32([2, 1]), 64, sinks=1, recent=8, lens_out=lens, count_out=count, weights_out=w_out)
    torch.cuda.synchronize()
    after = state(c, pool, w)
    for k in ("lens", "count", "w", "table"):
        assert torch.equal(before[k], after[k])
    assert lens.tolist() == [-3, -3, 64] and count.tolist() == want["count"].tolist()
    assert same(after["k"], want["k"]) and same(after["free"], want["free"])
    ph = c.block_table[2, :2].long()
    assert torch.equal(w_out[ph].cpu(), want["w"][ph.cpu()])
    w_out[ph] = -3.0
    assert bool((w_out == -3.0).all())
    # the same weights give the same keys again
    B.evict_q8(c, pool, w, i32([2, 1]), 64, sinks=1, recent=8, lens_out=lens, count_out=count, weights_out=w_out)
    assert torch.equal(w_out[ph].cpu(), want["w"][ph.cpu()])


def test_a_list_that_would_overflow_is_flagged():
    c, pool = make("int8", [300], P=32, spare=0)
    pool.free_count.fill_(c.cfg.num_phys_pages - 2)
    B.evict_q8(c, pool, spread_weights(c), i32([0]), 32)
    assert c.device_status() == B.DEV_CAPACITY and int(pool.free_count) == c.cfg.num_phys_pages
    assert c.seq_lens.tolist() == [32]


def test_many_slots_captured_and_on_another_stream():
    n = 1100  # more than a round of the planning
    lens = [20 + 7 * (i % 9) for i in range(n)]
    def once(how):
        c, pool = make("int8", lens, hkv=1, d=64, P=16, seed=6)
        w, ids = spread_weights(c), i32(list(range(n))[::-1])
        ws = B.alloc_evict_workspace(c, n, 40)
        torch.cuda.synchronize()
        before = state(c, pool, w)
        if how == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                B.evict_q8(c, pool, w, ids, 40, sinks=2, recent=5, workspace=ws)
            assert torch.equal(state(c, pool, w)["lens"], before["lens"])
            graph.replay()
        else:
            side = torch.cuda.Stream()
            B.evict_q8(c, pool, w, ids, 40, sinks=2, recent=5, workspace=ws, stream=side)
            side.synchronize()
        torch.cuda.synchronize()
        return c, before, state(c, pool, w), ids.tolist()
    c, before, a, ids = once("stream")
    _, _, b, _ = once("graph")
    want = expect(c, before, "int8", ids, 40, 40, 2, 5)
    for k in a:
        assert torch.equal(a[k], b[k]), k
        assert same(a[k], want[k]), k


def test_a_call_on_slots_that_stay_changes_nothing():
    c, pool = make("e4m3", [10, 64], P=16)
    w = spread_weights(c)
    before = state(c, pool, w)
    B.evict_q8(c, pool, w, i32([0, 1]), 64)
    B.evict_q8(c, pool, w, torch.zeros(0, dtype=torch.int32, device="cuda"), 64)
    after = state(c, pool, w)
    assert all(torch.equal(before[k], after[k]) for k in before) and c.device_status() == 0


@pytest.mark.parametrize("n_long,keep", [(1, 4100), (19, 4100), (20, 4100), (30, 900)])
def test_few_and_many_long_ones_among_many_slots(n_long, keep):
    """Clusters where few are evicted, blocks alone where many are: which of them is known on the device only."""
    lens = [keep + 60 + 7 * i if i < n_long else 30 + i for i in range(32)]
    c, pool = make("e4m3", lens, hkv=1, d=64, P=32, seed=3)
    check(c, pool, spread_weights(c), "e4m3", list(range(32))[::-1], keep, sinks=2, recent=40)


def test_idle_slots_are_not_looked_at():
    c, pool = make("int8", [300, 300, 300], P=32)
    B.evict_q8(c, pool, spread_weights(c), i32([0, 77, 0, 2]), 64, count=i32([1, 0, 0, 5]))
    assert c.device_status() == 0 and c.seq_lens.tolist() == [64, 300, 64]
