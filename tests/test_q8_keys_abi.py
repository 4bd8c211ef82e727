"""Refusals of differential attention, key weights and eviction, without a GPU
(pointers are dummies that are never dereferenced)."""

import contextlib
import ctypes

import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

from test_q8_abi import P256, cfg, lib  # noqa: F401

VIEW = B.Q8CacheView(*([P256] * 6), None)
BATCH = (None, P256, P256, 2, 2, 1)
ROWS = (P256, 4096, 128)


def diff(lib, c=None, batch=BATCH, score=None, lam=P256, stride=0, gain=None, eps=1e-5, ws=P256, ws_bytes=1 << 50,
         q=ROWS, out=ROWS, view=VIEW):
    return lib.entmaxkv_attend_diff_q8(c or cfg(), view, B.BatchView(*batch), B.RowsView(*q), score, lam, stride, gain, eps,
                                       ws, ws_bytes, B.RowsView(*out), None, None)


def weigh(lib, c=None, batch=BATCH, score=None, alpha=1.0, tau=P256, decay=1.0, weights=P256, ws=P256,
          ws_bytes=1 << 50, q=ROWS, view=VIEW):
    return lib.entmaxkv_weigh_q8(c or cfg(), view, B.BatchView(*batch), B.RowsView(*q), tau, score, alpha, None, decay,
                                 None, weights, ws, ws_bytes, None)


def evict(lib, c=None, view=VIEW, weights=P256, ids=P256, n=2, keep=100, above=100, sinks=4, recent=10, w_out=P256,
          lens=P256, free=P256, ws=P256, ws_bytes=1 << 50):
    return lib.entmaxkv_evict_q8(c or cfg(), view, weights, ids, None, n, keep, above, sinks, recent, w_out, lens, free, P256,
                                 P256, ws, ws_bytes, None)


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 96, 2), ("page_size", 8, 2), ("group", 9, 2), ("kv_dtype", B.BF16, 1), ("num_kv_heads", 0, 1),
    ("max_pages_per_seq", (1 << 25) + 1, 2)])
def test_bad_configs(lib, field, value, code):  # noqa: F811
    c = cfg(**{field: value})
    assert diff(lib, c) == code and weigh(lib, c) == code and evict(lib, c) == code
    assert lib.entmaxkv_weigh_q8_workspace(c, 1, 1, 1, 1.0) == 0 and lib.entmaxkv_evict_q8_workspace(c, 1, 1) == 0


def test_bad_difference_arguments(lib):  # noqa: F811
    assert diff(lib, cfg(group=3)) == 2 and diff(lib, cfg(group=1)) == 2       # heads without a partner
    assert diff(lib, lam=None) == 1 and diff(lib, stride=-1) == 1
    assert diff(lib, gain=P256, eps=0.0) == 1 and diff(lib, gain=P256, eps=float("nan")) == 1
    assert diff(lib, gain=P256, eps=-1.0) == 1 and diff(lib, gain=P256, eps=float("inf")) == 1
    assert diff(lib, ws=None) == 3 and diff(lib, ws=P256 + 8) == 3 and diff(lib, ws_bytes=1000) == 3
    assert diff(lib, score=B.ScoreView(-1.0, 0.0, 0)) == 1 and diff(lib, score=B.ScoreView(0.0, 1e-45, 0)) == 1
    assert diff(lib, out=(P256, 0, 128)) == 1 and diff(lib, q=(P256 + 2, 4096, 128)) == 1
    assert diff(lib, batch=(None, P256, P256, 0, 0, 0), lam=None) == 0         # nothing to do
    assert diff(lib, batch=(None, None, P256, 2, 2, 1)) == 1


def test_bad_weigh_arguments(lib):  # noqa: F811
    assert weigh(lib, tau=None) == 1 and weigh(lib, weights=None) == 1
    for d in (-0.5, float("nan"), float("inf")):
        assert weigh(lib, decay=d) == 1
    assert weigh(lib, alpha=0.5) == 1 and weigh(lib, alpha=float("nan")) == 1
    assert weigh(lib, alpha=1.5, batch=(None, P256, P256, 2, 4, 2)) == 2        # entmax: one row a sequence
    assert weigh(lib, ws=None) == 3 and weigh(lib, ws=P256 + 8) == 3 and weigh(lib, ws_bytes=0) == 3
    assert weigh(lib, score=B.ScoreView(0.0, 0.0, -1)) == 1 and weigh(lib, q=(P256, 4097, 128)) == 1
    assert weigh(lib, batch=(None, P256, P256, 2, 0, 1), tau=None) == 0
    assert weigh(lib, view=B.Q8CacheView(P256 + 8, *([P256] * 5), None)) == 1
    assert lib.entmaxkv_weigh_q8_workspace(cfg(), 2, 2, 1, 1.0) > 0
    assert lib.entmaxkv_weigh_q8_workspace(cfg(), 2, 4, 2, 1.5) == 0


def test_bad_evict_arguments(lib):  # noqa: F811
    assert evict(lib, n=0) == 0
    assert evict(lib, n=-1) == 1 and evict(lib, n=70000) == 1
    assert evict(lib, keep=0) == 1 and evict(lib, keep=3201, above=3201) == 1   # a row of the table holds 3200
    assert evict(lib, above=99) == 1                                            # below keep
    assert evict(lib, sinks=-1) == 1 and evict(lib, recent=-1) == 1 and evict(lib, sinks=91, recent=10) == 1
    assert evict(lib, sinks=0x7fffffff, recent=0x7fffffff) == 1
    assert evict(lib, ids=None) == 1 and evict(lib, lens=None) == 1 and evict(lib, free=None) == 1
    assert evict(lib, weights=None) == 1 and evict(lib, w_out=None) == 1 and evict(lib, weights=P256 + 8) == 1
    assert evict(lib, cfg(num_phys_pages=(1 << 27) + 1)) == 2                   # places are counted in 32 bits
    assert evict(lib, ws=None) == 3 and evict(lib, ws=P256 + 4) == 3 and evict(lib, ws_bytes=4096) == 3
    assert evict(lib, view=B.Q8CacheView(P256, P256, None, *([P256] * 3), None)) == 1
    f = lib.entmaxkv_evict_q8_workspace
    assert f(cfg(), 2, 100) >= 2 * 8 * 100 * 4 and f(cfg(), -1, 100) == 0 and f(cfg(), 2, 0) == 0


def z(*s, dt=torch.int32):
    return torch.zeros(*s, dtype=dt)


def small(group=4):
    pool, scale = z(4, 2, 16, 64, dt=torch.int8), z(4, 2, dt=torch.float32)
    return B.QuantCache.of(pool, pool.clone(), scale, scale.clone(), z(1, 4), z(1), group), B.Batch(z(1), z(1), 2, 2)


def test_binding_checks_its_tensors():
    c, batch = small()
    f = torch.float32
    q, lam, tau, w = z(2, 8, 64, dt=torch.bfloat16), z(4, dt=f), z(2, 8, dt=f), z(4, 2, 16, dt=f)
    pool = B.PagePool(z(4), z(1))
    odd, _ = small(3)
    bad = [lambda: B.attend_diff_q8(c, q, lam.double(), batch), lambda: B.attend_diff_q8(c, q, z(8, dt=f), batch),
           lambda: B.attend_diff_q8(c, q, z(2, 8, dt=f), batch), lambda: B.attend_diff_q8(c, q, z(3, 4, dt=f), batch),
           lambda: B.attend_diff_q8(odd, z(2, 6, 64, dt=torch.bfloat16), z(3, dt=f), batch),
           lambda: B.attend_diff_q8(c, q, lam, batch, gain=z(32, dt=f)),
           lambda: B.attend_diff_q8(c, q, z(2, 8, dt=f)[:, ::2], batch),
           lambda: B.weigh_q8(c, w, q, tau.half(), batch), lambda: B.weigh_q8(c, w, q, z(2, 4, dt=f), batch),
           lambda: B.weigh_q8(c, z(4, 2, 32, dt=f), q, tau, batch), lambda: B.weigh_q8(c, w, q, tau, batch, coef=z(2, dt=f)),
           lambda: B.weigh_q8(c, w, q, tau, batch, fresh=z(2)), lambda: B.weigh_q8(c, w, q[:1], tau, batch),
           lambda: B.evict_q8(c, pool, w.double(), z(1), 8), lambda: B.evict_q8(c, pool, w, z(1, dt=torch.int64), 8),
           lambda: B.evict_q8(c, B.PagePool(z(3), z(1)), w, z(1), 8),
           lambda: B.evict_q8(c, pool, w, z(1), 8, count=z(2)), lambda: B.evict_q8(c, pool, w, z(1), 8, lens_out=z(2)), lambda: B.evict_q8(c, pool, w, z(1), 8, count_out=z(2)),
           lambda: B.evict_q8(c, pool, None, z(1), 8, sinks=8, weights_out=w),
           lambda: B.evict_q8(c, pool, w, z(1), 8, weights_out=w[:2])]
    for call in bad:
        with pytest.raises(B.EntmaxKVError):
            call()


def test_what_the_calls_allocate_is_their_streams(monkeypatch):
    """Outputs and workspaces that are not given are made on the stream of the call."""
    log, active = [], [None]

    @contextlib.contextmanager
    def stream(s):
        active.append(s)
        yield
        active.pop()

    class Stream:
        device_index, cuda_stream = -1, 77

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 4096 if "workspace" in name else 0

    c, batch = small()
    f = torch.float32
    q, lam, tau, w = z(2, 8, 64, dt=torch.bfloat16), z(4, dt=f), z(2, 8, dt=f), z(4, 2, 16, dt=f)
    pool = B.PagePool(z(4), z(1))
    ids = z(1)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append("kept"))
    monkeypatch.setattr(B, "lib", lambda: Lib())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    for name in ("empty", "zeros", "full"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, real=real, **kw: (log.append(active[-1]), real(*a, **kw))[1])
    s = Stream()
    B.attend_diff_q8(c, q, lam, batch, stream=s)
    assert log == [s] * 3 + ["kept"] * 2
    log.clear()
    B.weigh_q8(c, w, q, tau, batch, stream=s)
    B.evict_q8(c, pool, w, ids, 8, stream=s)
    assert log == [s, s]
    other = Stream()
    other.device_index = 3
    for call in (lambda: B.attend_diff_q8(c, q, lam, batch, stream=other), lambda: B.weigh_q8(c, w, q, tau, batch, stream=other),
                 lambda: B.evict_q8(c, pool, w, ids, 8, stream=other)):
        with pytest.raises(B.EntmaxKVError, match="stream"):
            call()
