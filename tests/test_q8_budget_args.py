"""What the Python side of evictions and budgets refuses, without a GPU."""

import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

from test_q8_keys_abi import small, z


@pytest.mark.parametrize("name", ["keep", "above", "sinks", "recent"])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 8, 2 ** 40 + 8, -2 ** 31 - 1, 2 ** 63 - 1])
def test_numbers_past_32_bits_are_refused(monkeypatch, name, value):
    """Their low bits are numbers that the call would take."""
    c, _ = small()
    calls = []

    class Lib:
        def __getattr__(self, f):
            return lambda *a: calls.append(f) or (4096 if "workspace" in f else 0)

    monkeypatch.setattr(B, "lib", lambda: Lib())
    args = dict(keep=8, above=16, sinks=2, recent=2, workspace=torch.zeros(4096, dtype=torch.uint8))
    args[name] = value
    with pytest.raises(B.EntmaxKVError, match="32 bits"):
        B.evict_q8(c, B.PagePool(z(4), z(1)), z(4, 2, 16, dt=torch.float32), z(1), **args)
    assert not calls
    if name == "keep" and value > 0:
        with pytest.raises(B.EntmaxKVError, match="32 bits"):
            B.alloc_evict_workspace(c, 1, value)


def test_a_step_takes_a_gain_with_factors_only():
    """(Attention of heads has no norm: the gain was left aside without a word.)"""
    c, _ = small()
    with pytest.raises(B.EntmaxKVError, match="gain"):
        B.QuantStep(c, B.PagePool(z(4), z(1)), 1, gain=torch.ones(64))
