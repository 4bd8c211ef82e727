"""One decode policy on one synthetic cache, repeated: the small cases that
kernel profiles are taken on.

    python -m sparse_entmax_attention_gb300.profile_case --policy softmax --tokens 262144

The cache has the 1M workload's shape (32 query heads over 8 KV heads,
d = 128, page 32, bf16 keys and values, bf16 metadata copies) at the given
length, filled through the library's own append. Each of --reps decodes is
preceded by a 512 MiB write, so every decode starts with cold L2, as in the
bench. Policies: gaussian, topk, softmax, softmax_topk, full, full_dense.

    python -m sparse_entmax_attention_gb300.profile_case --q8 chunk --tokens 8192 --new 2048

repeats a call on the 8-bit cache instead (int8 codes, 32 query heads over 8 KV
heads, d = 128, page 32, --seqs sequences of --tokens tokens of which the last
--new are the step's): append, read, decode (softmax of one token each), chunk
(softmax of --new tokens each, capped with --softcap) or entmax (one token each).
"""

from __future__ import annotations

import argparse

import torch

from . import binding as B
from . import runner, synth


def q8_case(args, flush) -> int:
    new = 1 if args.q8 in ("decode", "entmax") else args.new
    pages = args.seqs * -(-args.tokens // 32)
    cache = B.QuantCache(8, 4, 128, 32, args.seqs, pages // args.seqs, pages)
    cache.block_table.copy_(torch.randperm(pages, device="cuda").view_as(cache.block_table))
    cache.seq_lens.fill_(args.tokens)

    def batch(n):
        start = torch.arange(args.seqs, dtype=torch.int32, device="cuda") * n
        return B.Batch(start, torch.full_like(start, n), args.seqs * n, n)

    def rows(n, heads):
        return torch.randn(args.seqs * n, heads, 128, device="cuda").bfloat16()

    every, last = batch(args.tokens), batch(new)
    B.append_q8(cache, rows(args.tokens, 8), rows(args.tokens, 8), every)
    k, v, q = rows(new, 8), rows(new, 8), rows(new, 32)
    first = torch.full((args.seqs,), args.tokens - new, dtype=torch.int32, device="cuda")
    alpha = args.alpha if args.q8 == "entmax" else 1.0
    out, ws = B.alloc_attend_outputs(cache, last), B.alloc_attend_workspace(cache, last, alpha)
    for _ in range(args.reps):
        flush.fill_(1)
        if args.q8 == "append":
            B.append_q8(cache, k, v, last)
        elif args.q8 == "read":
            B.read_q8(cache, first, last, k, v)
        else:
            B.attend_q8(cache, q, last, alpha=alpha, softcap=args.softcap, workspace=ws, outputs=out)
    torch.cuda.synchronize()
    status = cache.device_status()
    print(f"{args.q8}: {args.reps} calls, {args.seqs} sequences of {args.tokens} tokens, {new} new, device status {status:#x}")
    return 0 if status == 0 else 1


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--policy", default="gaussian")
    ap.add_argument("--tokens", type=int, default=262144)
    ap.add_argument("--reps", type=int, default=4)
    ap.add_argument("--budget", type=int, default=2048, help="top-k budget in tokens")
    ap.add_argument("--alpha", type=float, default=1.5)
    ap.add_argument("--margin", type=float, default=0.5)
    ap.add_argument("--q8", choices=["append", "read", "decode", "chunk", "entmax"], help="a call on the 8-bit cache")
    ap.add_argument("--seqs", type=int, default=1)
    ap.add_argument("--new", type=int, default=2048)
    ap.add_argument("--softcap", type=float, default=0.0)
    args = ap.parse_args(argv)
    flush = torch.empty(128 << 20, dtype=torch.int32, device="cuda")
    if args.q8:
        return q8_case(args, flush)
    spec = synth.Spec("profile-gqa32x8-d128-p32-bf16", 32, 8, 128, 32, [args.tokens], torch.bfloat16,
                      args.alpha, n_needles=64, n_outliers=4)
    wl = runner.Workload(spec, device="cuda", meta_bf16=True)
    policy, flags = args.policy, 0
    if policy == "full_dense":
        policy, flags = "full", B.FLAG_DENSE_V
    budget = args.budget if policy in ("topk", "softmax_topk") else 0
    margin = args.margin if policy == "gaussian" else 0.0
    ws = B.alloc_workspace(wl.cache, 1, policy, budget)
    out = B.alloc_outputs(wl.cache, 1, policy, budget)
    for _ in range(args.reps):
        flush.fill_(1)
        B.decode(wl.cache, wl.q, args.alpha, policy, budget, margin, flags, workspace=ws, outputs=out)
    torch.cuda.synchronize()
    status = wl.cache.device_status() & ~B.DEV_CAND_OVERFLOW
    print(f"{args.policy}: {args.reps} decodes of a {args.tokens}-token cache, device status {status:#x}")
    return 0 if status == 0 else 1


if __name__ == "__main__":
    raise SystemExit(main())
