"""Differential attention, key weights and eviction on pages that lie behind the
first 4 GiB of their pools: the same bits as on pages in front."""

import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

from q8_cases import batch_of, filled, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [1, 40])
def test_far_pages_give_the_same_bits(count):
    hkv, g, d, P, L = 8, 2, 128, 32, 900
    near, q = filled("int8", [L], [count], hkv=hkv, g=g, d=d, P=P)
    used, pages = -(-L // P), (1 << 32) // (hkv * P * d) + 64
    pools = [torch.empty(pages, hkv, P, d, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.ones(pages, hkv, device="cuda") for _ in range(2)]
    to = torch.arange(pages - used, pages, device="cuda")
    at = near.block_table[0, :used].long()
    for far, src in zip(pools + scales, (near.k_pool, near.v_pool, near.k_scale, near.v_scale)):
        far[to] = src[at]
    far = B.QuantCache.of(*pools, *scales, to.int().view(1, -1).contiguous(), i32([L]), g)
    lam = torch.full((hkv * g // 2,), 0.4, device="cuda")
    batch, results = batch_of([count]), []
    for c in (near, far):
        o = B.attend_diff_q8(c, q, lam, batch)
        w = B.alloc_weights(c)
        B.weigh_q8(c, w, q, o.tau, batch)
        ph = c.block_table[0, :used].long()
        gathered = w[ph].clone()
        free = torch.zeros(c.cfg.num_phys_pages, dtype=torch.int32, device="cuda")
        pool = B.PagePool(free, i32([0]))
        B.evict_q8(c, pool, w, i32([0]), 300, sinks=4, recent=30)
        kept = ph[:-(-300 // P)]
        k, v = B.read_q8(c, i32([0]), batch_of([300]))
        freed = (pool.free_pages[:int(pool.free_count)].long()[:, None] == ph).int().argmax(1)
        results.append((o.out, o.tau, gathered, w[kept], k, v, c.k_scale[kept], c.v_scale[kept], freed, c.seq_lens))
        assert c.device_status() == 0
    for a, b in zip(*results):
        assert torch.equal(a, b)
