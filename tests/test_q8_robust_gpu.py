"""The 8-bit cache where it is used in ways that single calls in an empty
device do not show: clusters that start one by one, calls on other streams,
non-finite queries, long and dense supports, steps that ask for too much."""

import pytest
import torch

from sparse_entmax_attention_gb300 import binding as B

from q8_cases import batch_of, filled

pytestmark = pytest.mark.gpu


def test_entmax_clusters_that_start_beside_other_work_give_the_same_bits():
    """Blocks of a cluster find their multiprocessors taken by another stream's products."""
    c, q = filled("int8", [9000], [1], hkv=4, g=4)
    batch = batch_of([1])
    first = B.attend_q8(c, q, batch, alpha=1.5)
    ws, o = B.alloc_attend_workspace(c, batch, 1.5), B.alloc_attend_outputs(c, batch)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x = torch.randn(2048, 2048, device="cuda").bfloat16()
    torch.cuda.synchronize()
    for _ in range(40):
        with torch.cuda.stream(side):
            for _ in range(4):
                x @ x
        B.attend_q8(c, q, batch, alpha=1.5, workspace=ws, outputs=o)
        torch.cuda.current_stream().synchronize()
        assert torch.equal(o.out, first.out) and torch.equal(o.tau, first.tau)
    torch.cuda.synchronize()
    assert c.device_status() == 0
