"""Variants of the kernels of key weights and eviction that are chosen by size: weights of 9 to 32 rows a slot, and
selections of more keys than a block keeps in shared memory."""

import re

import pytest
import torch

from test_cluster_order import CSRC
from test_q8_evict_gpu import check, make, spread_weights
from test_q8_weigh_gpu import filled, run

pytestmark = pytest.mark.gpu


def constant(file, name):
    with open(f"{CSRC}/{file}") as fh:
        return int(re.search(rf"\b{name} = (\d+);", fh.read()).group(1))


def masks(counts, lens, g):
    first = [(L - n + i if i % 5 else L) if i % 3 == 2 else max(0, L - n + i - 40)
             for L, n in zip(lens, counts) for i in range(n)]
    gen = torch.Generator(device="cuda").manual_seed(2)
    coef = torch.randn(sum(counts), 2 * g, generator=gen, device="cuda")  # half of them do not count
    slopes = torch.exp2(-torch.arange(1, 2 * g + 1, device="cuda").float())
    return ({}, {"softcap": 20.0, "window": 90, "decay": 0.5}, {"prefix": [30, 0, 5, 2][:len(counts)], "window": 8},
            {"first_key": first, "fresh": [100, 2000, 0, 1][:len(counts)]},
            {"slopes": slopes, "softcap": 8.0, "coef": coef},
            {"decay": 0.0, "fresh": [0, 0, 0, 0][:len(counts)], "scale": 0.01})


# rows of the largest slot, g times its count: two 8-row tiles for 9 to 16 rows, four for 17 to 32 (a block of half as
# many warps), both for softmax alone; the limit is kWeighRows
@pytest.mark.parametrize("code,d,P", [("int8", 128, 32), ("int8", 128, 16), ("e4m3", 128, 32), ("e4m3", 128, 16),
                                      ("int8", 64, 32), ("int8", 64, 16), ("e4m3", 64, 32), ("e4m3", 64, 16)])
@pytest.mark.parametrize("g,counts", [(3, [3, 1, 0, 2]), (8, [2, 1, 2, 0]),                     # 9, 16
                                      (1, [17, 5, 0, 9]), (8, [3, 1, 0, 2]), (5, [5, 2, 1, 3]),  # 17, 24, 25
                                      (7, [4, 3, 0, 1]), (4, [8, 7, 1, 2]), (1, [32, 1, 20, 0])])  # 28, 32, 32
def test_few_rows_a_slot(code, d, P, g, counts):
    assert 8 < g * max(counts) <= constant("q8.cuh", "kWeighRows") == 32
    lens = [max(1, n + x) for n, x in zip(counts, (500, 3, 1000, 0))]
    c, q = filled(code, lens, counts, hkv=2, g=g, d=d, P=P, seed=7)
    for kw in masks(counts, lens, g):
        run(c, q, counts, **kw)


@pytest.mark.parametrize("code,d,P,g,counts,lens", [("int8", 128, 32, 8, [4, 1], [40000, 7]),
                                                    ("e4m3", 64, 16, 1, [30, 30], [25000, 9001])])
def test_few_rows_on_many_tiles_a_warp(code, d, P, g, counts, lens):
    c, q = filled(code, lens, counts, hkv=2, g=g, d=d, P=P, seed=9)
    run(c, q, counts)
    run(c, q, counts, window=5000, decay=0.5)


def stepped(c, seed):
    """Weights of a few dozen values: the edge has many equals, over all blocks."""
    return torch.floor(2.0 * torch.log2(1.0 + spread_weights(c, seed, ties=0.2))) / 4.0


@pytest.mark.parametrize("code,P,keep", [("int8", 32, 4000), ("e4m3", 16, 30000)])
def test_a_cluster_reads_weights_again(code, P, keep):
    """One pair of more keys than a cluster of eight blocks keeps."""
    held = constant("q8_evict.cu", "kEvictKeys")
    c, pool = make(code, [8 * held + 5003, 20], hkv=1, d=64, P=P, seed=2)
    check(c, pool, stepped(c, 1), code, [1, 0], keep, sinks=3, recent=64)


@pytest.mark.parametrize("code,d,P,ties", [("int8", 64, 32, True), ("e4m3", 64, 16, False), ("e4m3", 128, 32, True)])
def test_blocks_alone_read_weights_again(code, d, P, ties):
    """Nine pairs and more with so few keys kept are a block each: of more keys than it keeps, of just as many, and
    of fewer."""
    held = constant("q8_evict.cu", "kEvictKeys")
    c, pool = make(code, [held + 1, 2 * held + 77, held, 1500], hkv=3, d=d, P=P, seed=4)
    w = stepped(c, 2) if ties else spread_weights(c, 2)
    check(c, pool, w, code, [2, 0, 3, 1], 900, sinks=2, recent=40)
