"""Runs one operation of the path a few times, for profilers (ncu) to capture.

    python -m gated_block_sparse_gate_b200.profile_cases --case train_fwd --reps 3
    python -m gated_block_sparse_gate_b200.profile_cases --case train_bwd --reps 3
    python -m gated_block_sparse_gate_b200.profile_cases --case train_bwd --workload train_bf16_n32768
    python -m gated_block_sparse_gate_b200.profile_cases --case sparse_fwd --topk 16 --reps 3
    python -m gated_block_sparse_gate_b200.profile_cases --case sparse_bwd --topk 16 --seq 16384
    python -m gated_block_sparse_gate_b200.profile_cases --case decode --batch 8 --reps 3
    python -m gated_block_sparse_gate_b200.profile_cases --case decode_grouped --batch 8
    python -m gated_block_sparse_gate_b200.profile_cases --case kv4_decode --batch 16 --seq 65536
    python -m gated_block_sparse_gate_b200.profile_cases --case kv4_decode_grouped --batch 16 --seq 65536
    python -m gated_block_sparse_gate_b200.profile_cases --case kv4_append --seq 32768
    python -m gated_block_sparse_gate_b200.profile_cases --case kv4_read --seq 32768
    python -m gated_block_sparse_gate_b200.profile_cases --case rope_fwd --seq 16384
    python -m gated_block_sparse_gate_b200.profile_cases --case rope_bwd --seq 16384

Inputs are the seeded workloads of ``inputs.py`` (optionally cut down with
--seq / --batch so a capture stays small); every launch goes through the C ABI. The 4-bit
cache and the rotary step take random values in the shapes of those workloads.
"""
from __future__ import annotations

import argparse
import dataclasses

import torch

from . import binding as gb
from .build import build
from .inputs import WORKLOADS, make_decode_inputs, make_prefill_inputs


def kv4_case(case, B, L, topk, reps, dev):
    """Decode of B sequences over random codes, or one prompt of L tokens appended and read back."""
    Hq, Hkv, d = 32, 8, 128
    g = torch.Generator(device=dev).manual_seed(1)
    if case in ("kv4_append", "kv4_read"):
        cache = gb.kv4_cache(1, Hkv, d, L=L, device=dev)
        start = torch.zeros(1, dtype=torch.int32, device=dev)
        K, V = torch.randn(2, 1, Hkv, L, d, generator=g, device=dev).to(torch.bfloat16)
        for _ in range(reps):
            gb.kv4_append(K, V, cache, start)
            if case == "kv4_read":
                gb.kv4_read(cache, start, L, dtype=torch.float32)
        return
    grouped = case == "kv4_decode_grouped"
    cache = gb.kv4_cache(B, Hkv, d, L=L, device=dev)
    for codes, params in (cache[:2], cache[2:]):
        codes.random_(0, 256, generator=g)
        params[..., 0].uniform_(0.2, 0.35, generator=g)
        params[..., 1].uniform_(-2.6, -1.6, generator=g)
    q = torch.randn(B, Hq, d, generator=g, device=dev).to(torch.bfloat16)
    S = 2 ** 0.5 * torch.randn(B, Hkv if grouped else Hq, -(-L // 64), generator=g, device=dev)
    for _ in range(reps):
        gb.kv4_decode(q, cache, S, L, topk=topk, group_shared=grouped)


def rope_case(case, N, reps, dev):
    """The packed projection of N tokens, 32 + 8 + 8 heads of 128."""
    g = torch.Generator(device=dev).manual_seed(1)
    split = (32, 8, 8)
    qkv, grads = torch.randn(2, 1, N, sum(split), 128, generator=g, device=dev).to(torch.bfloat16)
    q, k, v = qkv.split(split, 2)
    side = (*gb.rope_tables(N, 128, device=dev), torch.arange(N, dtype=torch.int32, device=dev)[None])
    w = torch.ones(2, 128, device=dev)
    out = gb.qkv_rope(q, k, v, *side, *w)
    for _ in range(reps):
        if case == "rope_bwd":
            gb.qkv_rope_backward(q, k, *side, *out, *w, grads=grads.split(split, 2))
        else:
            gb.qkv_rope(q, k, v, *side, *w, out=out)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--case", required=True, choices=("train_fwd", "train_bwd", "sparse_fwd",
                                                      "sparse_bwd", "decode", "decode_grouped",
                                                      "kv4_decode", "kv4_decode_grouped", "kv4_append",
                                                      "kv4_read", "rope_fwd", "rope_bwd"))
    ap.add_argument("--reps", type=int, default=3)
    ap.add_argument("--seq", type=int, default=None, help="override N (prefill) or L (decode)")
    ap.add_argument("--batch", type=int, default=None, help="override B (decode)")
    ap.add_argument("--topk", type=int, default=None)
    ap.add_argument("--workload", default=None, help="training workload (default train_bf16_n8192)")
    args = ap.parse_args(argv)
    build()
    gb.load_library()
    dev = torch.device("cuda", 0)
    if args.case.startswith("kv4_"):
        w = WORKLOADS["sparse_decode_bf16_b64_l131072"]
        kv4_case(args.case, args.batch or 16, args.seq or 65536, args.topk or w.topk[0], args.reps, dev)
    elif args.case.startswith("rope_"):
        rope_case(args.case, args.seq or 16384, args.reps, dev)
    elif args.case in ("decode", "decode_grouped"):
        w = WORKLOADS["sparse_decode_bf16_b64_l131072"]
        B = args.batch or w.B
        L = args.seq or w.N
        w = dataclasses.replace(w, B=B, N=L)
        x = make_decode_inputs(w, device=dev)
        k = args.topk or w.topk[0]
        S = x["S"]
        if args.case == "decode_grouped":  # one score row per kv group
            g = torch.Generator().manual_seed(w.seed + 1)
            S = (torch.randn(B, w.Hkv, w.Nb, generator=g) * 2 ** 0.5).to(dev)
        for _ in range(args.reps):
            gb.decode_ex(x["q"], x["Kc"], x["Vc"], S, L, topk=k,
                         group_shared=args.case == "decode_grouped")
    else:
        sparse = args.case in ("sparse_fwd", "sparse_bwd")
        w = WORKLOADS["sparse_prefill_bf16_n65536" if sparse else
                      (args.workload or "train_bf16_n8192")]
        if args.seq:
            w = dataclasses.replace(w, N=args.seq)
        bwd = args.case in ("train_bwd", "sparse_bwd")
        x = make_prefill_inputs(w, with_grad=bwd)
        d = {k: v.to(dev) for k, v in x.items()}
        mode = "sparse" if sparse else "train"
        k = (args.topk or w.topk[0]) if mode == "sparse" else 0
        O, LSE = gb.forward(d["Q"], d["K"], d["V"], d["S"], mode=mode, topk=k)
        for _ in range(args.reps):
            if bwd:
                gb.backward(d["Q"], d["K"], d["V"], d["S"], O, LSE, d["dO"], mode=mode, topk=k)
            else:
                gb.forward(d["Q"], d["K"], d["V"], d["S"], mode=mode, topk=k, out=O, lse=LSE)
    torch.cuda.synchronize()
    print("ok", args.case)


if __name__ == "__main__":
    main()
