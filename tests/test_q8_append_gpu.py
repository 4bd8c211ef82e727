"""The quantising append against the oracle, code for code, and its read-back."""

import numpy as np
import pytest
import torch

from oracle import q8 as oq
from sparse_entmax_attention_gb300 import binding as B

from q8_cases import DT, batch_of, empty_cache, i32

pytestmark = pytest.mark.gpu


class Mirror:
    """The oracle's copy of a cache's codes and scales, page by page."""

    def __init__(self, c, code):
        self.c, self.code = c, code
        n, hkv, P, d = c.k_pool.shape
        self.codes = {s: np.zeros((n, hkv, P, d)) for s in "kv"}
        self.scale = {s: np.zeros((n, hkv)) for s in "kv"}
        self.touched = set()

    def append(self, seq, old, k, v):
        P, table, odd = self.c.cfg.page_size, self.c.block_table[seq].tolist(), False
        for side, x in (("k", k), ("v", v)):
            x = x.double().cpu().numpy()
            at = 0
            while at < len(x):
                pos = old + at
                n_old = pos % P
                m = min(P - n_old, len(x) - at)
                ph = table[pos // P]
                self.touched.add(ph)
                for h in range(x.shape[1]):
                    self.codes[side][ph, h], self.scale[side][ph, h], o = oq.append_page(
                        self.codes[side][ph, h], self.scale[side][ph, h], n_old, x[at:at + m, h], self.code)
                    odd |= o
                at += m
        return odd

    def check(self):
        for side, pool, scale in (("k", self.c.k_pool, self.c.k_scale), ("v", self.c.v_pool, self.c.v_scale)):
            t = sorted(self.touched)
            assert np.array_equal(scale[t].double().cpu().numpy(), self.scale[side][t])
            assert np.array_equal(pool.float().double().cpu().numpy()[t], self.codes[side][t])


def _rows(total, hkv, d, seed, loud=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(total, hkv, d, generator=g, device="cuda") * loud
    return (x * torch.exp(torch.randn(total, hkv, 1, generator=g, device="cuda"))).bfloat16()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d,P", [(128, 32), (128, 16), (64, 32), (64, 16)])
def test_append_matches_the_oracle(code, d, P):
    # (old, new): from empty to several pages, over and up to page ends, into partly filled pages
    pairs = [(0, 1), (0, P), (0, 3 * P + 5), (1, 1), (P - 1, 1), (P - 1, 2), (P, 1), (5, 2 * P), (0, 0), (2 * P + 3, P)]
    old, new = [a for a, _ in pairs], [b for _, b in pairs]
    c = empty_cache(code, [a + b for a, b in pairs], hkv=3, d=d, P=P, seed=P + d)
    m = Mirror(c, code)
    c.seq_lens.copy_(i32(old))
    for part, counts, lens in ((0, old, old), (1, new, [a + b for a, b in pairs])):
        c.seq_lens.copy_(i32(lens))
        k, v = _rows(sum(counts), 3, d, 10 + part, 1.0 + part), _rows(sum(counts), 3, d, 20 + part)
        B.append_q8(c, k, v, batch_of(counts))
        at = 0
        for b, n in enumerate(counts):
            assert not m.append(b, lens[b] - n, k[at:at + n], v[at:at + n])
            at += n
    m.check()
    untouched = sorted(set(range(c.cfg.num_phys_pages)) - m.touched)
    assert untouched and not c.k_pool.float()[untouched].any() and not c.v_scale[untouched].any()
    assert c.device_status() == 0 and c.seq_lens.tolist() == [a + b for a, b in pairs]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_token_by_token_growth_requantises(code):
    c = empty_cache(code, [40], hkv=2, d=64, P=16)
    m = Mirror(c, code)
    k, v = _rows(40, 2, 64, 3), _rows(40, 2, 64, 4)
    k *= torch.linspace(0.1, 3.0, 40, device="cuda")[:, None, None].bfloat16()  # most tokens raise the scale
    for t in range(40):
        c.seq_lens.fill_(t + 1)
        B.append_q8(c, k[t:t + 1], v[t:t + 1], B.Batch.uniform(1))
        m.append(0, t, k[t:t + 1], v[t:t + 1])
    m.check()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_values_on_ties_and_both_signs(code):
    """Rows whose largest value makes the scale 2^-k exactly: quotients fall on ties."""
    g = oq.grid(code)
    ties = np.concatenate([(g[:-1] + g[1:]) / 2, g])
    ties = torch.tensor(ties[: 2 * 64]).bfloat16()
    x = torch.zeros(4, 1, 64)
    x[0, 0, :], x[1, 0, :] = ties[:64].float(), -ties[:64].float()
    x[2, 0, :], x[3, 0, :] = ties[64:128].float(), -ties[64:128].float()
    x[0, 0, 0] = oq.TOP[code]
    c = empty_cache(code, [4], hkv=1, d=64, P=16)
    m = Mirror(c, code)
    xs = (x * 2.0 ** -5).bfloat16().cuda()
    B.append_q8(c, xs, -xs, batch_of([4]))
    m.append(0, 0, xs, -xs)
    assert float(m.scale["k"][c.block_table[0, 0].item(), 0]) == 2.0 ** -5
    m.check()


def test_tiny_zero_and_huge_values():
    c = empty_cache("int8", [16, 16, 16, 16], hkv=1, d=64, P=16)
    m = Mirror(c, "int8")
    x = _rows(64, 1, 64, 9)
    x[16:32] = 0
    x[32:48] *= 2.0 ** -120
    x[48:64] = (x[48:64].float() * 1e37).bfloat16()
    B.append_q8(c, x, x, batch_of([16] * 4))
    for b in range(4):
        m.append(b, 0, x[16 * b:16 * b + 16], x[16 * b:16 * b + 16])
    m.check()
    assert c.device_status() == 0


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_infinities_and_nan_are_flagged(code):
    c = empty_cache(code, [7], hkv=2, d=128, P=16)
    m = Mirror(c, code)
    k, v = _rows(7, 2, 128, 1), _rows(7, 2, 128, 2)
    k[2, 1, 5], k[3, 1, 6], k[4, 0, 7] = float("inf"), float("-inf"), float("nan")
    B.append_q8(c, k, v, batch_of([7]))
    assert m.append(0, 0, k, v)
    m.check()
    assert c.device_status() == B.DEV_NONFINITE
    c2 = empty_cache(code, [1], hkv=2, d=128, P=16)
    nan = torch.full((1, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.append_q8(c2, nan, nan, batch_of([1]))
    assert not c2.k_pool.float().any() and float(c2.k_scale.max()) == 2.0 ** -96


def test_stale_scale_and_codes_of_a_reused_page_do_not_matter():
    for code in ("int8", "e4m3"):
        a = empty_cache(code, [20], hkv=2, d=128, P=16, garbage=True)
        b = empty_cache(code, [20], hkv=2, d=128, P=16)
        k, v = _rows(20, 2, 128, 1), _rows(20, 2, 128, 2)
        for c in (a, b):
            B.append_q8(c, k, v, batch_of([20]))
        ph = a.block_table[0, :2].long()
        assert torch.equal(a.k_scale[ph], b.k_scale[ph]) and torch.equal(a.v_scale[ph], b.v_scale[ph])
        assert torch.equal(a.k_pool.view(torch.int8)[ph[0]], b.k_pool.view(torch.int8)[ph[0]])
        assert torch.equal(a.v_pool.view(torch.int8)[ph[1], :, :4], b.v_pool.view(torch.int8)[ph[1], :, :4])


def test_strided_rows_seq_ids_gaps_and_idle_slots():
    hkv, g, d, P = 2, 3, 64, 16
    c = empty_cache("e4m3", [9, 0, 30, 17], hkv=hkv, g=g, d=d, P=P)
    m = Mirror(c, "e4m3")
    counts, seqs, gap = [30, 0, 9, 17], [2, 99, 0, 3], 4
    batch = batch_of(counts, seqs, gap)
    fused = _rows(batch.total, (g + 2) * hkv, d, 5)
    k, v = fused[:, g * hkv:g * hkv + hkv], fused[:, g * hkv + hkv:]
    fused_nan = fused.clone()
    own = torch.zeros(batch.total, dtype=torch.bool, device="cuda")
    for b, n in enumerate(counts):
        s0 = batch.start[b].item()
        own[s0:s0 + n] = True
    fused_nan[~own] = float("nan")  # rows of no slot are not read
    B.append_q8(c, fused_nan[:, g * hkv:g * hkv + hkv], fused_nan[:, g * hkv + hkv:], batch)
    for b, n in enumerate(counts):
        s0 = batch.start[b].item()
        if n:
            m.append(seqs[b], 0, k[s0:s0 + n], v[s0:s0 + n])
    m.check()
    assert c.device_status() == 0


def test_bad_slots_are_flagged_and_skipped():
    c = empty_cache("int8", [8, 8, 8, 8, 8], hkv=1, d=64, P=16)
    k = _rows(40, 1, 64, 1)
    before = c.k_pool.clone()
    B.append_q8(c, k, k, B.Batch(i32([0, 33, -1, 0, 0]), i32([9, 8, 3, -2, 8]), 40, 8, i32([0, 1, 2, 3, 7])))
    assert torch.equal(before, c.k_pool) and c.device_status() == B.DEV_BAD_BATCH | B.DEV_BAD_SEQ_ID
    c.block_table[0, 0] = -1
    c.status.zero_()
    B.append_q8(c, k, k, B.Batch(i32([0, 8]), i32([8, 8]), 40, 8))
    assert c.device_status() == B.DEV_BAD_PAGE_TABLE and bool(c.k_pool.any())


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d,P", [(128, 32), (64, 16)])
def test_read_back(code, d, P):
    lens, hkv = [3 * P + 7, 1, 0, P], 3
    c = empty_cache(code, lens, hkv=hkv, d=d, P=P)
    k, v = _rows(sum(lens), hkv, d, 1), _rows(sum(lens), hkv, d, 2)
    B.append_q8(c, k, v, batch_of(lens))
    first, counts = [5, 0, 0, P - 1], [3 * P, 1, 0, 1]
    batch = batch_of(counts, gap=1)
    ko = torch.full((batch.total, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    B.read_q8(c, i32(first), batch, ko, vo)
    for out, pool, scale in ((ko, c.k_pool, c.k_scale), (vo, c.v_pool, c.v_scale)):
        want = torch.full_like(out, 7.0)
        for b, n in enumerate(counts):
            for i in range(n):
                t = first[b] + i
                ph = c.block_table[b, t // P].item()
                val = pool.view(torch.int8)[ph, :, t % P].view(pool.dtype).float() * scale[ph][:, None]
                want[batch.start[b].item() + i] = val.bfloat16()
        assert torch.equal(out, want)
    assert c.device_status() == 0
    B.read_q8(c, i32([8, 1, 0, -1]), batch_of([3 * P, 1, 0, 1]))
    assert c.device_status() == B.DEV_BAD_BATCH


def test_read_back_into_a_16_bit_cache():
    """A sequence handed over to the page-metadata cache: read_q8 in the layout that append takes."""
    T, hkv, d, P = 300, 2, 128, 16
    c = empty_cache("int8", [T], hkv=hkv, d=d, P=P)
    k, v = _rows(T, hkv, d, 1), _rows(T, hkv, d, 2)
    B.append_q8(c, k, v, batch_of([T]))
    ko, vo = (torch.empty(1, hkv, T, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.read_q8(c, i32([0]), batch_of([T]), ko[0].transpose(0, 1), vo[0].transpose(0, 1))
    full = B.PagedCache(hkv, 4, d, P, 1, 20, 20, torch.bfloat16)
    pool = B.PagePool.full(20)
    B.plan_pages(full, pool, i32([T]), B.alloc_plan(1, T), advance=False)  # append counts the tokens itself
    B.append(full, ko, vo)
    q = torch.randn(1, 8, d, device="cuda").bfloat16()
    a = B.decode(full, q, 1.5, "full")
    b = B.attend_q8(c, q.view(1, 8, d), B.Batch.uniform(1), alpha=1.5)
    torch.cuda.synchronize()
    assert full.device_status() == 0 and full.seq_lens.tolist() == [T]
    # the 16-bit cache holds each value rounded to bf16 (2^-8 relative): a score moves by at most
    # 2^-8·Σ|q||k|/√d, far above every other rounding here
    kk = ko[0].float().repeat_interleave(4, 0)
    mag = (q[0].float().abs()[:, None] * kk.abs()).sum(-1).max() / d ** 0.5
    assert float((a.tau - b.tau).abs().max()) <= float(2.0 ** -8 * mag * 0.5 * 2)
    torch.testing.assert_close(b.out.float(), a.out, rtol=0.1, atol=0.1)


@pytest.mark.parametrize("n", [300, 1100])
def test_many_slots_write_and_read_what_few_do(n):
    """One call for all slots and one for every 100 of them leave the same cache and read the same rows."""
    hkv, d, P = 2, 64, 16
    lens = [1 + (b * 11) % 70 for b in range(n)]
    k, v = _rows(sum(lens), hkv, d, 3), _rows(sum(lens), hkv, d, 4)
    one, many = (empty_cache("int8", lens, hkv=hkv, d=d, P=P) for _ in range(2))
    B.append_q8(one, k, v, batch_of(lens))
    ko, vo = B.read_q8(one, i32([0] * n), batch_of(lens))
    for b in range(0, n, 100):
        ids = list(range(b, min(b + 100, n)))
        a, z = sum(lens[:b]), sum(lens[:ids[-1] + 1])
        part = batch_of(lens[b:ids[-1] + 1], ids)
        B.append_q8(many, k[a:z], v[a:z], part)
        kp, vp = B.read_q8(many, i32([0] * len(ids)), part)
        assert torch.equal(ko[a:z], kp) and torch.equal(vo[a:z], vp)
    assert one.device_status() == 0 and many.device_status() == 0
    # quantised once, by half a step at most, and rounded to bf16 (2^-8 of up to 127 steps)
    assert (ko.float() - k.float()).abs().max() <= (0.5 + 127 / 256) * float(one.k_scale.max())
