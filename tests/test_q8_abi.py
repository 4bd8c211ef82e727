"""Refusals of the 8-bit cache's entry points, without a GPU (pointers are
dummies that are never dereferenced)."""

import ctypes
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


def cfg(**kw):
    base = dict(num_kv_heads=8, group=4, head_dim=128, page_size=32, max_seqs=4, max_pages_per_seq=100,
                num_phys_pages=400, kv_dtype=B.I8)
    base.update(kw)
    return B.Config(*[base[f] for f, _ in B.Config._fields_])


def attend(lib, c=None, view=None, batch=None, q=None, score=None, alpha=1.0, ws=P256, ws_bytes=1 << 50, out=None):
    c = c or cfg()
    view = view or B.Q8CacheView(*([P256] * 6), None)
    batch = batch or B.BatchView(None, P256, P256, 2, 2, 1)
    q = q or B.RowsView(P256, 4096, 128)
    out = out or B.RowsView(P256, 4096, 128)
    return lib.entmaxkv_attend_q8(c, view, batch, q, score, alpha, ws, ws_bytes, out, None, None)


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 96, 2), ("page_size", 8, 2), ("group", 9, 2), ("kv_dtype", B.BF16, 1), ("kv_dtype", 9, 1),
    ("num_kv_heads", 0, 1), ("num_kv_heads", 5000, 2), ("max_pages_per_seq", 0, 1), ("max_pages_per_seq", 1 << 30, 2),
    ("max_pages_per_seq", (1 << 25) + 1, 2)])
def test_bad_configs(lib, field, value, code):
    c = cfg(**{field: value})
    assert attend(lib, c) == code
    b, r, view = B.BatchView(None, P256, P256, 2, 2, 1), B.RowsView(P256, 1024, 128), B.Q8CacheView(*([P256] * 6), None)
    assert lib.entmaxkv_append_q8(c, view, b, r, r, None) == code
    assert lib.entmaxkv_read_q8(c, view, b, P256, r, r, None) == code
    assert lib.entmaxkv_attend_q8_workspace(c, 1, 1, 1, 1.0) == 0


def test_the_16_bit_calls_take_no_8_bit_cache(lib):
    view = B.CacheView(*([P256] * 8), None)
    p = ctypes.c_void_p(P256)
    assert lib.entmaxkv_append(ctypes.byref(cfg()), ctypes.byref(view), p, p, None, 1, 4, None) == 1


def test_bad_attend_arguments(lib):
    assert attend(lib, alpha=0.5) == 1 and attend(lib, alpha=float("nan")) == 1 and attend(lib, alpha=float("inf")) == 1
    assert attend(lib, alpha=1.5, batch=B.BatchView(None, P256, P256, 2, 4, 2)) == 2   # entmax: one token
    assert attend(lib, ws=P256 + 8) == 3 and attend(lib, ws=None) == 3 and attend(lib, ws_bytes=1000) == 3
    assert attend(lib, batch=B.BatchView(None, None, P256, 2, 2, 1)) == 1
    assert attend(lib, batch=B.BatchView(None, P256, P256, -1, 2, 1)) == 1
    assert attend(lib, batch=B.BatchView(None, P256, P256, 70000, 2, 1)) == 1
    assert attend(lib, batch=B.BatchView(None, P256, P256, 0, 0, 0)) == 0             # nothing to do
    assert attend(lib, batch=B.BatchView(None, P256, P256, 2, 0, 1)) == 0
    assert attend(lib, view=B.Q8CacheView(P256 + 8, *([P256] * 5), None)) == 1        # pools from 16 bytes
    assert attend(lib, view=B.Q8CacheView(P256, P256, None, *([P256] * 3), None)) == 1
    for rows in (B.RowsView(P256 + 2, 4096, 128), B.RowsView(P256, 4097, 128), B.RowsView(P256, 4096, 12),
                 B.RowsView(P256, -4096, 128), B.RowsView(None, 4096, 128)):
        assert attend(lib, q=rows) == 1 and attend(lib, out=rows) == 1
    assert attend(lib, out=B.RowsView(P256, 0, 128)) == 1                             # rows that are written
    for score in (B.ScoreView(-1.0, 0.0, 0), B.ScoreView(0.0, -1.0, 0), B.ScoreView(0.0, 0.0, -1),
                  B.ScoreView(float("nan"), 0.0, 0), B.ScoreView(0.0, float("inf"), 0), B.ScoreView(0.0, 1e-45, 0),
                  B.ScoreView(0.0, 1e19, 0), B.ScoreView(0.0, float("nan"), 0)):
        assert attend(lib, score=score) == 1


def test_calls_whose_tiles_pass_32_bits(lib):
    c = cfg(max_pages_per_seq=1 << 25, num_phys_pages=1 << 25)  # 2^30 tokens, 2^23 tiles of 128
    assert lib.entmaxkv_attend_q8_workspace(c, 1, 15000, 15000, 1.0) > 0          # 234 items and two
    assert lib.entmaxkv_attend_q8_workspace(c, 1, 17000, 17000, 1.0) == 0         # 265 and two
    assert attend(lib, c, batch=B.BatchView(None, P256, P256, 1, 17000, 17000)) == 2
    assert lib.entmaxkv_attend_q8_workspace(c, 1, 17000, 12, 1.0) > 0             # few tokens a slot: counted in 64 bits


def test_bad_plan_arguments(lib):
    def plan(c=None, n=2, total=4, table=P256, free=P256):
        return lib.entmaxkv_plan_pages(c or cfg(), table, P256, None, None, P256, n, total, free, P256, P256, None,
                                       P256, P256, None, None, None)
    assert plan(n=0) == 0 and plan(n=-1) == 1 and plan(n=70000) == 1 and plan(total=-1) == 1
    assert plan(table=None) == 1 and plan(free=None) == 1
    assert plan(cfg(page_size=24)) == 2 and plan(cfg(max_seqs=0)) == 1 and plan(cfg(max_pages_per_seq=1 << 30)) == 2
    rel = lib.entmaxkv_release_pages
    assert rel(cfg(), P256, P256, None, None, 0, P256, P256, None) == 0
    assert rel(cfg(), None, P256, None, None, 1, P256, P256, None) == 1
    assert rel(cfg(), P256, P256, None, None, -1, P256, P256, None) == 1


def test_workspace_sizes(lib):
    f = lib.entmaxkv_attend_q8_workspace
    assert f(cfg(), 16, 16, 1, 1.0) > 0 and f(cfg(), 16, 640, 40, 1.0) > f(cfg(), 16, 80, 5, 1.0)
    assert f(cfg(), 4, 4, 1, 1.5) >= 4 * 8 * 100 * 32 * 4 * 4       # a z for every token and head
    assert f(cfg(), -1, 4, 1, 1.0) == 0 and f(cfg(), 1, 4, 2, 1.5) == 0


def test_binding_checks_its_tensors():
    """Shapes, types and devices are checked before the library is called (CPU tensors here)."""
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)  # noqa: E731
    pool, scale = z(4, 2, 16, 64, dt=torch.int8), z(4, 2, dt=torch.float32)
    c = B.QuantCache.of(pool, pool.clone(), scale, scale.clone(), z(1, 4), z(1), 4)
    batch = B.Batch(z(1), z(1), 2, 2)
    rows = z(2, 2, 64, dt=torch.bfloat16)
    bad = [lambda: B.append_q8(c, rows.float(), rows, batch), lambda: B.append_q8(c, rows[:1], rows, batch),
           lambda: B.append_q8(c, rows, rows[..., ::2], batch),
           lambda: B.attend_q8(c, rows, batch), lambda: B.read_q8(c, z(2), batch),
           lambda: B.QuantCache.of(pool.float(), pool, scale, scale, z(1, 4), z(1), 4),
           lambda: B.QuantCache.of(pool, pool[:2], scale, scale, z(1, 4), z(1), 4),
           lambda: B.QuantCache.of(pool, pool, scale[:2], scale, z(1, 4), z(1), 4),
           lambda: B.QuantCache.of(pool, pool, scale, scale, z(1, 4, dt=torch.int64), z(1), 4),
           lambda: B.Batch(z(1), z(2), 2, 2), lambda: B.PagePool(z(4), z(2)),
           lambda: B.PageTable(z(2, 3), z(3), 16, 4)]
    for call in bad:
        with pytest.raises(B.EntmaxKVError):
            call()
