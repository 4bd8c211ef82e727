"""Tensors that a call given a stream makes itself are made on that stream (read
with a fake library and fake streams, without a GPU)."""

import contextlib

import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B


class FakeStream:
    device_index, cuda_stream = -1, 77


class FakeLib:
    def __getattr__(self, name):
        return lambda *a: 4096 if "workspace" in name else 0


@pytest.fixture
def seen(monkeypatch):
    """(function, stream it ran under) of every allocation, and of the library's calls."""
    log, active = [], [None]

    @contextlib.contextmanager
    def stream(s):
        active.append(s)
        yield
        active.pop()

    def watched(name):
        real = getattr(torch, name)

        def f(*a, **kw):
            log.append((name, active[-1]))
            return real(*a, **kw)
        return f

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream())
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("kept", None)))
    monkeypatch.setattr(B, "lib", lambda: FakeLib())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    for name in ("empty", "zeros", "full"):
        monkeypatch.setattr(torch, name, watched(name))
    return log


def z(*shape, dt=torch.int32):
    return torch.zeros(*shape, dtype=dt)


def q8():
    pool, scale = z(4, 2, 16, 64, dt=torch.int8), z(4, 2, dt=torch.float32)
    return B.QuantCache.of(pool, pool.clone(), scale, scale.clone(), z(1, 4), z(1), 4), B.Batch(z(1), z(1), 2, 2)


CALLS = {
    "attend_q8": lambda s: B.attend_q8(*[(c, z(2, 8, 64, dt=torch.bfloat16), b) for c, b in [q8()]][0], stream=s),
    "read_q8": lambda s: B.read_q8(*[(c, z(1), b) for c, b in [q8()]][0], stream=s),
    "decode": lambda s: B.decode(B.PagedCache(2, 4, 64, 16, 1, 4, 4, torch.bfloat16, "cpu"),
                                 z(1, 8, 64, dt=torch.bfloat16), policy="full", stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_allocates_is_its_streams(seen, name):
    s = FakeStream()
    made = {"attend_q8": 3, "read_q8": 2, "decode": 6}[name]
    kept = {"attend_q8": 2, "read_q8": 2, "decode": 5}[name]
    CALLS[name](s)
    allocs = [at for f, at in seen if f != "kept"]
    assert allocs[-made:] == [s] * made and sum(f == "kept" for f, _ in seen) == kept
    seen.clear()
    CALLS[name](None)  # on the current stream as ever
    assert all(at is None for _, at in seen) and not any(f == "kept" for f, _ in seen)


def test_given_tensors_are_left_where_they_are(seen):
    c, b = q8()
    o, ws = B.alloc_attend_outputs(c, b), z(4096, dt=torch.uint8)
    q = z(2, 8, 64, dt=torch.bfloat16)
    k = z(2, 2, 64, dt=torch.bfloat16)
    seen.clear()
    B.attend_q8(c, q, b, workspace=ws, outputs=o, stream=FakeStream())
    assert not seen
    got = B.read_q8(c, z(1), b, k, None, stream=FakeStream())
    assert got[0] is k and got[1] is not k and got[1].shape == k.shape
    got = B.read_q8(c, z(1), b, None, k, stream=FakeStream())
    assert got[1] is k and got[0] is not k


def test_a_stream_of_another_device_is_refused(seen):
    c, b = q8()
    other = FakeStream()
    other.device_index = 3
    with pytest.raises(B.EntmaxKVError, match="stream"):
        B.append_q8(c, z(2, 2, 64, dt=torch.bfloat16), z(2, 2, 64, dt=torch.bfloat16), b, stream=other)
