"""Order of accesses to shared memory that other blocks or warps write, read from the
kernels' source.

A block may write the shared memory of another block of its cluster only once
that block is known to run, which a cluster barrier shows; and a block may not
end while others still read from it."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_entmax_attention_gb300", "csrc")
REMOTE = re.compile(r"\bpeer\(|map_shared_rank\(")
BARRIER = re.compile(r"barrier\.cluster\.wait|\bcluster_sync\(\)|\bcluster\.sync\(\)")


def _kernels(text):
    """(name, body) of each __global__ function, comments taken out."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\s*\([^{;]*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[m.end():i]


def _remote_kernels():
    found = []
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, f)) as fh:
                found += [(f, name, body) for name, body in _kernels(fh.read()) if REMOTE.search(body)]
    return found


CASES = _remote_kernels()


def test_the_kernels_are_found():
    assert {name for _, name, _ in CASES} >= {"tauhat_kernel", "topk_cluster_kernel", "ent_finish_kernel"}


@pytest.mark.parametrize("name,body", [(n, b) for _, n, b in CASES], ids=[n for _, n, _ in CASES])
def test_a_barrier_comes_before_the_first_remote_access(name, body):
    first, barrier = REMOTE.search(body), BARRIER.search(body)
    assert barrier and barrier.start() < first.start(), name


def test_entmax_finish_ends_behind_a_barrier():
    body = next(b for _, n, b in CASES if n == "ent_finish_kernel")
    assert list(BARRIER.finditer(body))[-1].start() > list(REMOTE.finditer(body))[-1].start()


def test_page_facts_of_a_tile_are_handed_on_by_threads():
    """In the chunk kernel the converters' plain stores of page facts reach the softmax warps through the issuing
    thread: it waits for the converters' arrivals and then arrives itself, once a tile, at the barrier that the
    softmax warps wait for (a commit's arrival alone says nothing of another thread's stores)."""
    with open(os.path.join(CSRC, "q8_chunk.cuh")) as fh:
        body = dict((n, b) for n, b in _kernels(fh.read()))["chunk_kernel"]
    assert "mbar_init(&s_full[i][c], 1 + c)" in body
    assert body.count("tm_commit(&s_full") == 1 and "if (c == 1) mbar_arrive(&s_full[hf][1]);" in body
    assert body.index("meta[it & 3][") < body.index("mbar_arrive(&k_full[sg])") < body.index("wait_warp(&k_full[it & 1]")
