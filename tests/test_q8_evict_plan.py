"""The eviction's plan for more slots than a block has threads: its phases read from the source, and slots that are
refused, repeated or idle among more than a thousand."""

import numpy as np
import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

from test_cluster_order import CSRC, _kernels


def test_marks_of_bad_pages_are_read_behind_the_barrier_only():
    """Every block of the cluster numbers a round's pages for itself and takes its share of the numbers, so nothing that
    the numbering reads may be written by another block before the next cluster barrier."""
    with open(f"{CSRC}/q8_evict.cu") as fh:
        body = dict(_kernels(fh.read()))["evict_plan_kernel"]
    phases = body.split("cluster_sync();")
    writes = [i for i, p in enumerate(phases) if "a.bad[" in p]
    reads = [i for i, p in enumerate(phases) if "__ldcg(a.bad" in p]
    assert len(writes) == 2 and "a.bad[b] = 0" in phases[writes[0]]
    # a lambda stands where it is defined: one that reads the marks and is called in the pass that sets them counts
    assert reads and min(reads) > max(writes)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1100, 2300])
def test_refused_repeated_and_idle_slots_among_many(n):
    """Bad table entries in neighbouring slots and in far ones of a round, first, middle and last pages: each such slot
    stays as it was, and so do second namings and idle slots."""
    from q8_cases import i32
    from test_q8_evict_gpu import expect, make, same, spread_weights, state
    keep, P = 40, 16
    lens = [30 + 11 * (i % 13) for i in range(n)]
    c, pool = make("e4m3", lens, hkv=1, d=64, P=P, seed=n)
    w = spread_weights(c)
    rng = np.random.default_rng(n)
    bad = sorted(set(rng.choice(n, 60, replace=False).tolist()) | {0, 1, 2, 3, 500, 501, 1022, 1023, 1024, 1025, n - 1})
    table = c.block_table.cpu()
    for i, s in enumerate(bad):
        used = -(-lens[s] // P)
        table[s, (0, used - 1, used // 2)[i % 3]] = (c.cfg.num_phys_pages, -1, 2 ** 31 - 1)[i % 3]
    c.block_table.copy_(table)
    ids = rng.permutation(n).tolist()
    count = [1] * n
    for b in rng.choice(n, 50, replace=False).tolist():
        count[b] = 0
    idle = {ids[b] for b in range(n) if count[b] == 0}
    named = ids + ids[:40] + [n, -1, 2 ** 31 - 1, -2 ** 31]  # a second time, and nobody
    count += [3] * 40 + [1] * 4
    before = state(c, pool, w)
    order, seen = [], set()
    for s, k in zip(named, count):
        if k and 0 <= s < n and s not in seen:
            seen.add(s)
            order.append(s)
    want = expect(c, before, "e4m3", [s for s in order if s not in bad], keep, keep, 2, 5)
    for _ in range(3):  # (from the same state: blocks of the plan are never at the same place twice)
        for k, t in (("k", c.k_pool), ("v", c.v_pool)):
            t.view(torch.int8).copy_(before[k])
        for k, t in (("ks", c.k_scale), ("vs", c.v_scale), ("lens", c.seq_lens), ("w", w), ("free", pool.free_pages),
                     ("count", pool.free_count)):
            t.copy_(before[k])
        c.status.zero_()
        B.evict_q8(c, pool, w, i32(named), keep, sinks=2, recent=5, count=i32(count))
        torch.cuda.synchronize()
        got = state(c, pool, w)
        for k in got:
            if k in "kv":
                assert same(got[k].view(torch.float8_e4m3fn), want[k].view(torch.float8_e4m3fn)), k
            else:
                assert same(got[k], want[k]), k
        assert c.device_status() == B.DEV_BAD_SEQ_ID | B.DEV_BAD_PAGE_TABLE | B.DEV_BAD_BATCH
    assert idle and all(int(got["lens"][s]) == lens[s] for s in idle - seen)
