"""Differential attention over the 8-bit cache against the oracle."""

import numpy as np
import pytest
import torch

from oracle import q8 as oq
from sparse_entmax_attention_gb300 import binding as B

from q8_cases import batch_of, dense, filled, i32, v_scales

pytestmark = pytest.mark.gpu


def check_diff(c, q, counts, o, lam, gain=None, eps=1e-5, seq_ids=None, scale=0.0, softcap=0.0, slopes=None, window=0,
               prefix=None, first_key=None):
    """Compare rows with the oracle. Each map's output is good to e = (2^-11 p + small + 2δp)·|v| as for attention
    (check_attend), so a difference is to E = e0 + |λ|·e1 + 2^-21·(|o0| + |λ·o1|) (a quotient, a product, an FMA of
    2^-24 each, and λ/sum's two). With a norm, Σy² lies between Σ(|y|−E)₊² and Σ(|y|+E)², which bounds the value from
    both sides; 2^-20 for the norm's own fp32 sum, root and two products. Then half a step of bf16 (2^-8)."""
    G, d = c.cfg.group, c.cfg.head_dim
    out, tau = o.out.double().cpu().numpy(), o.tau.double().cpu().numpy()
    Q, sc = q.double().cpu().numpy(), scale if scale else d ** -0.5
    lam = lam.double().cpu().numpy()
    g = None if gain is None else gain.double().cpu().numpy()
    for b, n in enumerate(counts):
        if n == 0:
            continue
        seq = b if seq_ids is None else seq_ids[b]
        r0 = sum(counts[:b])
        fk = None if first_key is None else first_key[r0:r0 + n]
        for i in range(c.num_q_heads // 2):
            K, V = dense(c, seq, 2 * i // G, "k"), dense(c, seq, 2 * i // G, "v")
            s = v_scales(c, seq, 2 * i // G)
            ref, err = [], []
            for h in (2 * i, 2 * i + 1):
                sl = 0.0 if slopes is None else float(slopes[h])
                r, t, Pw, S = oq.attend(K, V, Q[r0:r0 + n, h], 1.0, scale, softcap, sl, window,
                                        0 if prefix is None else prefix[b], fk)
                mag = (np.abs(Q[r0:r0 + n, h]) @ np.abs(K).T).max(initial=0.0) * sc
                delta = 2.0 ** -20 * (mag + sl * len(K) + softcap + 1.0)
                small = 2.0 ** -33 * (Pw * s).max(1, initial=0.0)[:, None] * np.isfinite(S) / s
                ref.append(r)
                err.append((2.0 ** -11 * Pw + small + 2 * delta * Pw) @ np.abs(V))
                some = ~np.isnan(t)
                assert np.array_equal(np.isnan(tau[r0:r0 + n, h]), ~some), (b, h)
                te = np.abs(tau[r0:r0 + n, h] - t)[some]
                assert np.all(te <= 2 * delta + 2.0 ** -23 * np.abs(t[some])), (b, h)
            la = lam[i] * np.ones(n) if lam.ndim == 1 else lam[r0:r0 + n, i]
            y = oq.difference(*ref, la)
            E = err[0] + np.abs(la)[:, None] * err[1] + 2.0 ** -21 * (np.abs(ref[0]) + np.abs(la[:, None] * ref[1]))
            got = out[r0:r0 + n, i]
            if g is None:
                tol = E + 2.0 ** -8 * np.abs(y) + 1e-30
                assert np.all(np.abs(got - y) <= tol), (b, i, float((np.abs(got - y) / tol).max()))
            else:
                root = lambda x: 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)  # noqa: E731
                lo = np.where(y - E > 0, (y - E) * root(np.abs(y) + E), (y - E) * root(np.maximum(np.abs(y) - E, 0.0)))
                hi = np.where(y + E > 0, (y + E) * root(np.maximum(np.abs(y) - E, 0.0)), (y + E) * root(np.abs(y) + E))
                lo, hi = np.minimum(lo * g, hi * g), np.maximum(lo * g, hi * g)
                lo -= (2.0 ** -8 + 2.0 ** -20) * np.abs(lo) + 1e-30
                hi += (2.0 ** -8 + 2.0 ** -20) * np.abs(hi) + 1e-30
                assert np.all((got >= lo) & (got <= hi)), (b, i)
            assert not got[np.isnan(tau[r0:r0 + n, 2 * i])].any()


def factors(total, pairs, each, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.sigmoid(torch.randn((total, pairs) if each else (pairs,), generator=gen, device="cuda"))


def gains(d, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return 0.2 * torch.exp(0.3 * torch.randn(d, generator=gen, device="cuda"))


@pytest.mark.parametrize("code,d,P", [("int8", 128, 32), ("e4m3", 128, 16), ("int8", 64, 16), ("e4m3", 64, 32)])
@pytest.mark.parametrize("g", [2, 4, 6, 8])
@pytest.mark.parametrize("norm,each", [(False, False), (True, True)])
def test_single_rows(code, d, P, g, norm, each):
    lens = [1, 2, 33, 700, 5001]
    c, q = filled(code, lens, [1] * 5, hkv=2, g=g, d=d, P=P, seed=g)
    lam, gain = factors(5, g, each), gains(d) if norm else None
    o = B.attend_diff_q8(c, q, lam, batch_of([1] * 5), gain=gain)
    assert c.device_status() == 0
    check_diff(c, q, [1] * 5, o, lam, gain)


@pytest.mark.parametrize("code,d,P,g,counts", [
    ("int8", 128, 32, 4, [3, 1, 0, 2]), ("e4m3", 64, 16, 8, [6, 2, 1, 5]), ("int8", 64, 32, 6, [8, 7, 3, 1]),
    ("int8", 128, 16, 4, [70, 1, 130, 33]), ("e4m3", 128, 32, 6, [90, 0, 43, 20]), ("e4m3", 64, 16, 2, [200, 129, 1, 64]),
    ("int8", 64, 32, 8, [17, 300, 2, 1])])
@pytest.mark.parametrize("norm", [False, True])
def test_several_rows_with_masks(code, d, P, g, counts, norm):
    """Drafted tokens and chunks, with capped scores, slopes, windows, prefixes and rows that see nothing."""
    lens = [n + x for n, x in zip(counts, (500, 3, 1000, 0))]
    lens = [max(1, n) for n in lens]
    c, q = filled(code, lens, counts, hkv=2, g=g, d=d, P=P, seed=7)
    total = sum(counts)
    lam, gain = factors(total, g, True), gains(d) if norm else None
    first = [(L - n + i if i % 5 else L) if i % 3 == 2 else max(0, L - n + i - 40)
             for L, n in zip(lens, counts) for i in range(n)]
    slopes = torch.exp2(-torch.arange(1, 2 * g + 1, device="cuda").float())
    for kw in ({}, {"softcap": 20.0, "window": 90}, {"prefix": [30, 0, 5, 2]}, {"first_key": first},
               {"slopes": slopes, "softcap": 8.0}):
        call = {k: i32(v) if k in ("prefix", "first_key") else v for k, v in kw.items()}
        o = B.attend_diff_q8(c, q, lam, batch_of(counts), gain=gain, **call)
        assert c.device_status() == 0
        check_diff(c, q, counts, o, lam, gain, **kw)


@pytest.mark.parametrize("n,count,norm", [(70000, 1, True), (70000, 2, False), (40000, 60, True), (40000, 33, False)])
def test_long_sequences_joined_over_blocks(n, count, norm):
    c, q = filled("int8", [n, 50], [count, 1], hkv=2, g=2, d=64, P=32, seed=3)
    lam, gain = factors(count + 1, 2, False), gains(64) if norm else None
    o = B.attend_diff_q8(c, q, lam, batch_of([count, 1]), gain=gain)
    check_diff(c, q, [count, 1], o, lam, gain)


def test_rows_of_strided_tensors_and_rows_outside_the_batch():
    counts = [2, 1, 40]
    for most in (2, 40):
        cs = counts[:2] + [min(most, 40)]
        c, q = filled("int8", [100, 7, 300], cs, hkv=2, g=4, d=128, P=16)
        total = sum(cs) + 9
        wide = torch.full((total, 3, 8, 136), 7.0, device="cuda").bfloat16()
        wide[:sum(cs), 1, :, :128] = q
        out = torch.full((total, 2, 5, 128), 9.0, device="cuda").bfloat16()
        tau = torch.full((total, 8), 9.0, device="cuda")
        lam = factors(total, 4, True)
        batch = B.Batch(i32([0, 2, 3]), i32(cs), total, most)
        o = B.attend_diff_q8(c, wide[:, 1, :, :128], lam, batch, outputs=B.AttendOutputs(out[:, 1, :4], tau))
        check_diff(c, q, cs, B.AttendOutputs(o.out[:sum(cs)], tau[:sum(cs)]), lam)
        assert bool((out[:, 0] == 9).all() and (out[:, 1, 4] == 9).all() and (out[sum(cs):] == 9).all())
        assert bool((tau[sum(cs):] == 9).all())


def test_two_keys_a_pair_as_one_concatenated_row():
    """Maps with keys of their own of half the width: queries padded with zeros on either side."""
    L, d, counts = 300, 128, [1, 20]
    c, _ = filled("int8", [L, L], counts, hkv=2, g=2, d=d, P=32, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(1)
    half = torch.randn(21, 4, d // 2, generator=gen, device="cuda").bfloat16()
    q = torch.zeros(21, 4, d, device="cuda", dtype=torch.bfloat16)
    q[:, 0::2, :64], q[:, 1::2, 64:] = half[:, 0::2], half[:, 1::2]
    lam = factors(21, 2, False)
    o = B.attend_diff_q8(c, q, lam, batch_of(counts), scale=64 ** -0.5)
    check_diff(c, q, counts, o, lam, scale=64 ** -0.5)
    K, V, x = dense(c, 1, 0, "k"), dense(c, 1, 0, "v"), half.double().cpu().numpy()
    maps = [oq.attend(K[:, 64 * m:64 * m + 64], V, x[1:, m])[0] for m in (0, 1)]
    assert np.allclose(oq.difference(*maps, float(lam[0]) * np.ones(20)), o.out[1:, 0].double().cpu().numpy(), atol=0.02)


def test_a_non_finite_query_stays_in_its_pair():
    for count in (1, 40):
        c, q = filled("e4m3", [200], [count], hkv=2, g=4, d=64, P=16)
        lam = factors(count, 4, False)
        want = B.attend_diff_q8(c, q, lam, batch_of([count]), gain=gains(64))
        q = q.clone()
        q[0, 3, 5] = float("inf")
        o = B.attend_diff_q8(c, q, lam, batch_of([count]), gain=gains(64))
        assert bool(o.out[0, 1].isnan().all()) and bool(o.tau[0, 3].isnan())
        o.out[0, 1], o.tau[0, 3] = want.out[0, 1], want.tau[0, 3]
        assert torch.equal(o.out, want.out) and torch.equal(o.tau, want.tau)


def test_equal_maps_cancel():
    """Both queries of a pair alike and a factor of 1: exactly zero, with a norm too."""
    for count in (1, 50):
        c, q = filled("int8", [900], [count], hkv=2, g=4, d=128, P=32)
        q = q.clone()
        q[:, 1::2] = q[:, 0::2]
        for gain in (None, gains(128)):
            o = B.attend_diff_q8(c, q, torch.ones(4, device="cuda"), batch_of([count]), gain=gain)
            assert not bool(o.out.any()) and torch.equal(o.tau[:, 0::2], o.tau[:, 1::2])


def test_a_bad_page_is_flagged_and_its_keys_are_not_there():
    c, q = filled("int8", [100], [1], hkv=1, g=2, d=64, P=16)
    c.block_table[0, 2] = 10 ** 6
    o = B.attend_diff_q8(c, q, factors(1, 1, False), batch_of([1]))
    assert c.device_status() == B.DEV_BAD_PAGE_TABLE and bool(o.out.isfinite().all())


def test_captured_and_on_another_stream():
    c, q = filled("int8", [3000, 10, 400], [1, 1, 1], hkv=2, g=4, d=128, P=32)
    lam, gain, batch = factors(3, 4, True), gains(128), batch_of([1, 1, 1])
    want = B.attend_diff_q8(c, q, lam, batch, gain=gain)
    ws, o = B.alloc_attend_workspace(c, batch), B.alloc_diff_outputs(c, batch)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    B.attend_diff_q8(c, q, lam, batch, gain=gain, workspace=ws, outputs=o, stream=side)
    side.synchronize()
    assert torch.equal(o.out, want.out) and torch.equal(o.tau, want.tau)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.attend_diff_q8(c, q, lam, batch, gain=gain, workspace=ws, outputs=o)
    for _ in range(2):
        o.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.out, want.out)
