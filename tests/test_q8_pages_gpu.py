"""Page planning and release on the device against the host oracle (all
outputs are whole numbers: equality)."""

import random

import pytest
import torch

from oracle import q8 as oq
from sparse_entmax_attention_gb300 import binding as B

from q8_cases import i32

pytestmark = pytest.mark.gpu


def _case(seed, n, max_new, P, spare, bad=False):
    rng = random.Random(seed)
    max_seqs, max_pages = n + 3, 9
    lens = [rng.choice([0, 0, 1, P - 1, P, P + 1, rng.randrange(0, 5 * P)]) for _ in range(max_seqs)]
    held = [-(-x // P) for x in lens]
    num = sum(held) + spare
    ids = list(range(num))
    rng.shuffle(ids)
    table, at = [], 0
    for m in held:
        table.append(ids[at:at + m] + [-1] * (max_pages - m))
        at += m
    free = ids[at:]
    seqs = rng.sample(range(max_seqs), n)
    new = [rng.choice([0, 1, rng.randrange(0, max_new + 1)]) for _ in range(n)]
    if bad:
        new[0], seqs[1], new[1], new[2] = -3, max_seqs, 5, max_pages * P + 1
        seqs[3] = -1 if new[3] == 0 else seqs[3]  # an idle slot's row is not looked at
    return lens, table, P, num, free, seqs, new


def _run(lens, table, P, num, free, seqs, new, total, in_place):
    t = B.PageTable(i32(table), i32(lens), P, num)
    stack = torch.full((num,), -7, dtype=torch.int32, device="cuda")
    stack[:len(free)] = i32(free)
    pool = B.PagePool(stack, i32([len(free)]))
    plan = B.alloc_plan(len(seqs), total)
    lens_out = None if in_place else t.seq_lens.clone()
    count_out = None if in_place else i32([-1])
    B.plan_pages(t, pool, i32(new), plan, seq_ids=i32(seqs), lens_out=lens_out, count_out=count_out)
    torch.cuda.synchronize()
    return t, pool, plan, t.seq_lens if in_place else lens_out, pool.free_count if in_place else count_out


@pytest.mark.parametrize("n,max_new,P,spare,bad", [
    (1, 1, 16, 1, False), (5, 40, 16, 30, False), (5, 40, 32, 4, False), (64, 3, 32, 40, False),
    (300, 60, 16, 200, True), (1500, 30, 16, 900, False), (2100, 9, 32, 0, True)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_the_oracle(n, max_new, P, spare, bad, in_place):
    lens, table, P, num, free, seqs, new = _case(n * 7 + spare, n, max_new, P, spare, bad)
    total = sum(max(x, 0) for x in new) + 11
    want = oq.plan(lens, table, P, num, free, seqs, new, total)
    t, pool, plan, lens_out, count = _run(lens, table, P, num, free, seqs, new, total, in_place)
    tab, wl, wf, start, cnt, pos, slots, refused = want
    assert t.block_table.tolist() == tab and lens_out.tolist() == wl and count.item() == len(wf)
    assert plan.start.tolist() == start and plan.count.tolist() == cnt
    used = [i for i, p in enumerate(pos) if p is not None]
    assert [plan.positions[i].item() for i in used[:200]] == [pos[i] for i in used[:200]]
    p, s = plan.positions.tolist(), plan.slots.tolist()
    assert all(p[i] == (-1 if pos[i] is None else pos[i]) for i in range(total))  # rows behind: as they were (-1)
    assert all(s[i] == (-1 if slots[i] is None else slots[i]) for i in range(total))
    assert (t.device_status() != 0) == bool(refused)
    assert pool.free_pages[:len(free)].tolist() == free


def test_rows_behind_the_last_token_and_a_short_total():
    t = B.PageTable(i32([[-1] * 4] * 2), i32([0, 0]), 16, 8)
    pool = B.PagePool.full(8)
    plan = B.alloc_plan(2, 20)
    plan.positions.fill_(77)
    plan.slots.fill_(77)
    B.plan_pages(t, pool, i32([5, 3]), plan)
    assert plan.positions.tolist() == [0, 1, 2, 3, 4, 0, 1, 2] + [77] * 12
    assert plan.slots.tolist() == [0, 1, 2, 3, 4, 16, 17, 18] + [77] * 12 and t.device_status() == 0
    # the second slot's rows leave the arrays: refused, its pages stay free
    t2 = B.PageTable(i32([[-1] * 4] * 2), i32([0, 0]), 16, 8)
    pool2 = B.PagePool.full(8)
    plan2 = B.alloc_plan(2, 6)
    B.plan_pages(t2, pool2, i32([5, 3]), plan2)
    assert plan2.count.tolist() == [5, 0] and pool2.free_count.item() == 7
    assert t2.device_status() == B.DEV_BAD_BATCH and t2.seq_lens.tolist() == [5, 0]
    assert plan2.positions.tolist() == [0, 1, 2, 3, 4, -1]


def test_plan_without_advancing_and_without_maps():
    t = B.PageTable(i32([[-1] * 4]), i32([3]), 16, 8)
    t.block_table[0, 0] = 6
    pool = B.PagePool(i32([0, 1, 2, 3, 4, 5, 7, -1]), i32([7]))
    plan = B.alloc_plan(1, 40)
    B.plan_pages(t, pool, i32([40]), plan, advance=False)
    assert t.seq_lens.tolist() == [3] and t.block_table.tolist() == [[6, 7, 5, -1]] and pool.free_count.item() == 5


def test_release_gives_back_what_planning_took():
    P, num = 16, 64
    t = B.PageTable(i32([[-1] * 12] * 5), i32([0] * 5), P, num)
    pool = B.PagePool.full(num)
    plan = B.alloc_plan(5, 400)
    B.plan_pages(t, pool, i32([100, 1, 0, 33, 16]), plan)
    table, height = t.block_table.clone(), pool.free_count.item()
    before = pool.free_pages.clone()
    B.release_pages(t, pool, i32([3]))
    assert t.seq_lens.tolist() == [100, 1, 0, 0, 16] and pool.free_count.item() == height + 3
    B.plan_pages(t, pool, i32([33]), B.alloc_plan(1, 33), seq_ids=i32([3]))
    assert torch.equal(t.block_table, table) and pool.free_count.item() == height
    # a sequence named twice gives its pages back once; bad rows are flagged
    B.release_pages(t, pool, i32([4, 4, 0, 1, 3, 2]))
    assert pool.free_count.item() == num and sorted(pool.free_pages.tolist()) == list(range(num))
    assert t.device_status() == 0 and before.numel() == num
    B.release_pages(t, pool, i32([9, -1]))
    assert t.device_status() == B.DEV_BAD_SEQ_ID and pool.free_count.item() == num


def test_release_drops_bad_entries_and_stops_at_a_full_list():
    t = B.PageTable(i32([[2, 99, -4, 1], [0, 3, 5, 6]]), i32([64, 64]), 16, 7)
    pool = B.PagePool(i32([4, -1, -1, -1, -1, -1, -1]), i32([1]))
    B.release_pages(t, pool, i32([0]))
    assert pool.free_count.item() == 3 and pool.free_pages[:3].tolist() == [4, 1, 2]
    assert t.device_status() == B.DEV_BAD_PAGE_TABLE
    pool = B.PagePool(i32([4, 1, 2, 0, 3, -1, -1]), i32([5]))
    B.release_pages(t, pool, i32([1]))
    assert pool.free_count.item() == 7 and t.device_status() == B.DEV_BAD_PAGE_TABLE | B.DEV_CAPACITY
