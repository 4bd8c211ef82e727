"""What attention over the 8-bit cache refuses beside bad arguments, without a GPU."""

import os

import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

P256 = 256


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from sparse_entmax_attention_gb300 import build
        build.build_library()
    return B.lib()


def cfg(pages=100):
    return B.Config(8, 4, 128, 32, 4, pages, 400, B.I8)


def test_bounded_planning_checks_its_arguments(lib):
    def plan(max_count, n=2, table=P256):
        return lib.entmaxkv_plan_pages_bounded(cfg(), table, P256, None, None, P256, n, 4, max_count, P256, P256, P256,
                                               None, P256, P256, None, None, None)
    assert plan(-1) == 1 and plan(3, table=None) == 1 and plan(3, n=-1) == 1 and plan(3, n=0) == 0


@pytest.mark.parametrize("alpha,pages,fine", [
    (1.0, 100, True), (1.0 + 2.0 ** -10, 100, True), (1.0 + 2.0 ** -11, 100, False), (1.25, 1 << 25, True),
    (4.0, 1 << 25, True), (5.5, 1 << 25, False),      # 2^30 keys: up to order 5
    (8.0, 4096, True), (8.1, 4096, False), (11.0, 100, True), (12.0, 100, False)])
def test_orders_that_cannot_be_solved_are_refused(lib, alpha, pages, fine):
    c = cfg(pages)
    size = lib.entmaxkv_attend_q8_workspace(c, 1, 1, 1, alpha)
    assert (size > 0) == fine
    view, batch = B.Q8CacheView(*([P256] * 6), None), B.BatchView(None, P256, P256, 0, 0, 1)  # no slot: nothing is queued
    rows = B.RowsView(P256, 4096, 128)
    code = lib.entmaxkv_attend_q8(c, view, batch, rows, None, alpha, P256, 1 << 50, rows, None, None)
    assert code == (0 if fine else 2)


@pytest.mark.parametrize("n,count", [(0, 1), (1, 1), (3, 0), (5, 4)])
def test_a_uniform_batch_has_every_slot(n, count):
    b = B.Batch.uniform(n, count, device="cpu")
    assert b.start.tolist() == [i * count for i in range(n)] and b.count.tolist() == [count] * n
    assert (b.total, b.max_count, b.view.n_seqs) == (n * count, count, n)
    assert b.start.dtype == b.count.dtype == torch.int32
