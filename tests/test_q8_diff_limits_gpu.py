"""Differences of pairs whose values are far from 1, and of maps that are nearly alike."""

import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

from q8_cases import batch_of, filled
from test_q8_diff_gpu import check_diff, factors, gains

pytestmark = pytest.mark.gpu

# single tokens (whole units, pieces joined in a block, and over blocks), drafted tokens, chunks (whole and joined)
SHAPES = [([700, 40], [1, 1]), ([70000, 5], [1, 1]), ([70000, 900], [2, 1]), ([600, 300], [40, 9]), ([40000, 50], [60, 7])]


@pytest.mark.parametrize("lens,counts", SHAPES)
@pytest.mark.parametrize("code,d,power", [("int8", 64, 80), ("e4m3", 128, 100), ("int8", 128, 63), ("e4m3", 64, -80)])
def test_a_norm_of_values_whose_squares_pass_fp32(code, lens, counts, d, power):
    """One sequence's V rows are 2^power times as large as the others': its normalised rows are those of the cache
    as it was but for ε, and the other sequences' are untouched."""
    c, q = filled(code, lens, counts, hkv=2, g=4, d=d, P=32, seed=11)
    lam, gain = factors(sum(counts), 4, True), gains(d)
    batch = batch_of(counts)
    plain = B.attend_diff_q8(c, q, lam, batch, gain=gain).out.clone()
    pages = c.block_table[0, :-(-lens[0] // 32)].long()
    c.v_scale[pages] *= 2.0 ** power
    o = B.attend_diff_q8(c, q, lam, batch, gain=gain)
    check_diff(c, q, counts, o, lam, gain)
    assert torch.equal(o.out[counts[0]:], plain[counts[0]:])
    assert bool(o.out[:counts[0]].isfinite().all()) and c.device_status() == 0


@pytest.mark.parametrize("lens,counts", SHAPES)
@pytest.mark.parametrize("code,d,norm", [("int8", 128, False), ("e4m3", 64, True)])
@pytest.mark.parametrize("apart", [2.0 ** -3, 2.0 ** -8])
def test_maps_that_are_nearly_alike(code, lens, counts, d, norm, apart):
    """Second queries are the first ones but for a part, and factors next to 1: the difference is small beside both
    maps, and its error stays that of their weights' 11 bits (which is what check_diff allows, before the norm)."""
    c, q = filled(code, lens, counts, hkv=2, g=4, d=d, P=32, seed=12)
    q = q.clone()
    gen = torch.Generator(device="cuda").manual_seed(5)
    q[:, 1::2] = q[:, 0::2] * (1.0 + apart * torch.randn(q[:, 0::2].shape, generator=gen, device="cuda"))
    lam = 1.0 - 2.0 ** -6 * factors(sum(counts), 4, True)
    gain = gains(d) if norm else None
    o = B.attend_diff_q8(c, q, lam, batch_of(counts), gain=gain)
    check_diff(c, q, counts, o, lam, gain)
    assert c.device_status() == 0


@pytest.mark.parametrize("lens,counts", SHAPES)
def test_equal_calls_give_equal_bits(lens, counts):
    c, q = filled("e4m3", lens, counts, hkv=2, g=4, d=128, P=16, seed=13)
    lam, gain, batch = factors(sum(counts), 4, True), gains(128), batch_of(counts)
    want = B.attend_diff_q8(c, q, lam, batch, gain=gain)
    busy = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for i in range(10):
        busy.fill_(i)
        o = B.attend_diff_q8(c, q, lam, batch, gain=gain)
        assert torch.equal(o.out, want.out) and torch.equal(o.tau, want.tau)
