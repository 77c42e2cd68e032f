"""Runs one case of the library's operations on seeded synthetic inputs and prints
its CUDA-event time per call -- a quick check of a build, and the command the
profiles are taken with.

    python -m fp4_fp8_quant_gb300 prepare --tokens 4632 [--repeat 3] [--route auto|small|pair]
    python -m fp4_fp8_quant_gb300 quant --rows 4632 --cols 7168 [--repeat 3]
    python -m fp4_fp8_quant_gb300 indexer --queries 4632 --keys 4632 [--topk 2048] [--full] [--repeat 3]
    python -m fp4_fp8_quant_gb300 attend --tokens 4632 [--past 0] [--q-heads 64] [--kv-heads 1] [--topk 2048] [--repeat 3]
    python -m fp4_fp8_quant_gb300 experts --tokens 4632 [--experts 64] [--k 8] [--dim 7168] [--hidden 2048] [--repeat 3]
    python -m fp4_fp8_quant_gb300 adapt --requests 64 [--length 1] [--adapters 48] [--rank 64] [--dim 7168] [--out-dim 8192] [--repeat 3]

`prepare` calls iq_prepare_q on the prefill workload when --tokens is 4632
(positions 0..M-1) and on the decode workload otherwise (random positions);
`quant` calls the FP8 1x128 quantizer on the blocks workload; `indexer` scores
random FP4 queries against a random FP4 key cache (causal unless --full) and
selects the top-k keys per query; `attend` is one attention layer of a step over
the paged 8-bit cache: it writes the new tokens' keys and values, scores and
selects keys with the indexer, attends to the selected keys, and for comparison
to all of them, and reads the tokens back; `experts` is the feed-forward block of
gated experts (routing, quantised rows, first and second product, combination on
top of the token's row) and each of its steps alone; `adapt` adds the adapters of
--requests requests of --length rows each to a projection's output.  L2 is flushed
before every call.
"""

from __future__ import annotations

import argparse
import sys

import numpy as np
import torch

from . import iq
from . import workloads as W


def _bf16(bits: np.ndarray, dev) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(dev)


def _time_calls(fn, repeat: int, dev) -> list[float]:
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=dev)
    out = []
    for _ in range(repeat):
        flush.fill_(1)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        fn()
        b.record()
        torch.cuda.synchronize()
        out.append(a.elapsed_time(b) * 1e3)
    return out


def _attend(args, dev) -> None:
    T, past, page, D, H = args.tokens, args.past, 64, 128, args.kv_heads
    n = past + T
    pages = -(-n // page)
    gen = torch.Generator(device=dev).manual_seed(1)

    def normal(rows, heads):
        return torch.randn((rows, heads, D), generator=gen, device=dev, dtype=torch.float32).to(torch.bfloat16)

    def lengths(first, last):                        # one sequence whose newest tokens are [first, last)
        return (torch.tensor([0, last - first], dtype=torch.int32, device=dev),
                torch.tensor([last], dtype=torch.int32, device=dev))

    cache = iq.KVCache.empty(pages, H, page, D, dev)
    table = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)[None]
    if past:
        iq.kv_cache_write(cache, normal(past, H), normal(past, H), table, *lengths(0, past))
    batch = (table, *lengths(past, n))
    k, v, q = normal(T, H), normal(T, H), normal(T, args.q_heads)
    q4, qs, k4, ks, w, visible = (torch.from_numpy(a).to(dev) for a in W.indexer_inputs(T, n, seed=1, causal=True))
    logits = torch.empty((T, n), dtype=torch.float32, device=dev)
    idx = torch.empty((T, args.topk), dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    work = torch.empty(max(1, iq.kv_attention_workspace_bytes(T, args.q_heads, H, D)), dtype=torch.uint8, device=dev)
    steps = [
        ("write", lambda: iq.kv_cache_write(cache, k, v, *batch)),
        ("indexer logits", lambda: iq.indexer_logits(q4, qs, k4, ks, w, visible, logits=logits)),
        (f"top-{args.topk}", lambda: iq.indexer_topk(logits, visible, args.topk, indices=idx)),
        ("attention, selected keys", lambda: iq.kv_attention_topk(cache, q, idx, *batch, out=out, workspace=work)),
        ("attention, all keys", lambda: iq.kv_attention(cache, q, *batch, out=out, workspace=work)),
        ("read", lambda: iq.kv_cache_read(cache, T, *batch, k=k, v=v)),
    ]
    print(f"attend T={T} past={past} heads={args.q_heads}/{H} (us per call)")
    for name, fn in steps:
        print(f"  {name}: " + " ".join(f"{u:.2f}" for u in _time_calls(fn, args.repeat, dev)))


def _random_weights(gen, dev, *shape):
    """E4M3 codes of either sign below 2 (finite), and scales that keep a product's size."""
    codes = torch.randint(0, 0x40, shape, generator=gen, device=dev, dtype=torch.uint8)
    codes |= torch.randint(0, 2, shape, generator=gen, device=dev, dtype=torch.uint8) << 7
    G, N, K = shape
    exponent = 127 - int(np.ceil(np.log2(K) / 2))
    return codes, torch.full((G, -(-N // 128), K // 128), exponent, dtype=torch.uint8, device=dev)


def _experts(args, dev) -> None:
    gen = torch.Generator(device=dev).manual_seed(1)
    T, E, k, K, I = args.tokens, args.experts, args.k, args.dim, args.hidden
    x = torch.randn((T, K), generator=gen, device=dev).to(torch.bfloat16)
    logits = torch.randn((T, E), generator=gen, device=dev)
    up, up_sf = _random_weights(gen, dev, E, 2 * I, K)
    down, down_sf = _random_weights(gen, dev, E, K, I)

    def block():
        r = iq.moe_route(logits, k, normalize=True)
        h = iq.grouped_gemm(*iq.fp8_quant_1x128_ue8m0(x, rows=r.rows), up, up_sf, r.row_start, gated=True)
        y = iq.grouped_gemm(*iq.fp8_quant_1x128_ue8m0(h), down, down_sf, r.row_start)
        return iq.moe_combine(y, r.slots, r.weights, add=x)

    r = iq.moe_route(logits, k, normalize=True)
    xq, xs = iq.fp8_quant_1x128_ue8m0(x, rows=r.rows)
    h = iq.grouped_gemm(xq, xs, up, up_sf, r.row_start, gated=True)
    hq, hs = iq.fp8_quant_1x128_ue8m0(h)
    y = iq.grouped_gemm(hq, hs, down, down_sf, r.row_start)
    for name, fn in (("block", block), ("route", lambda: iq.moe_route(logits, k, normalize=True)),
                     ("quantised rows", lambda: iq.fp8_quant_1x128_ue8m0(x, rows=r.rows)),
                     ("first product", lambda: iq.grouped_gemm(xq, xs, up, up_sf, r.row_start, gated=True)),
                     ("quantised hidden rows", lambda: iq.fp8_quant_1x128_ue8m0(h)),
                     ("second product", lambda: iq.grouped_gemm(hq, hs, down, down_sf, r.row_start)),
                     ("combination", lambda: iq.moe_combine(y, r.slots, r.weights, add=x))):
        us = _time_calls(fn, args.repeat, dev)
        print(f"experts T={T} {k} of {E}, {K} x {I}: {name} " + " ".join(f"{u:.2f}" for u in us) + " us per call")


def _adapt(args, dev) -> None:
    gen = torch.Generator(device=dev).manual_seed(1)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(torch.bfloat16)

    R, A, T = args.requests, args.adapters, args.requests * args.length
    x, base = normal(T, args.dim), normal(T, args.out_dim)
    a, b = normal(A, args.rank, args.dim, scale=args.dim ** -0.5), normal(A, args.out_dim, args.rank, scale=args.rank ** -0.5)
    scale = torch.ones(A, device=dev)
    row_start = torch.arange(0, T + 1, args.length, dtype=torch.int32, device=dev)
    adapter = (torch.arange(R, device=dev) % A).to(torch.int32)
    us = _time_calls(lambda: iq.adapters(x, base, a, b, scale, row_start, adapter), args.repeat, dev)
    print(f"adapt {R} requests of {args.length} rows, {A} adapters of rank {args.rank}, {args.dim} -> {args.out_dim}: "
          + " ".join(f"{u:.2f}" for u in us) + " us per call")


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(prog="python -m fp4_fp8_quant_gb300")
    sub = ap.add_subparsers(dest="cmd", required=True)
    p = sub.add_parser("prepare")
    p.add_argument("--tokens", type=int, default=4632)
    p.add_argument("--repeat", type=int, default=3)
    p.add_argument("--route", choices=["auto", "small", "pair"], default="auto")
    q = sub.add_parser("quant")
    q.add_argument("--rows", type=int, default=4632)
    q.add_argument("--cols", type=int, default=7168)
    q.add_argument("--repeat", type=int, default=3)
    ix = sub.add_parser("indexer")
    ix.add_argument("--queries", type=int, default=4632)
    ix.add_argument("--keys", type=int, default=4632)
    ix.add_argument("--topk", type=int, default=2048)
    ix.add_argument("--full", action="store_true")
    ix.add_argument("--repeat", type=int, default=3)
    at = sub.add_parser("attend")
    at.add_argument("--tokens", type=int, default=4632)
    at.add_argument("--past", type=int, default=0)
    at.add_argument("--q-heads", type=int, default=64)
    at.add_argument("--kv-heads", type=int, default=1)
    at.add_argument("--topk", type=int, default=2048)
    at.add_argument("--repeat", type=int, default=3)
    ex = sub.add_parser("experts")
    ex.add_argument("--tokens", type=int, default=4632)
    ex.add_argument("--experts", type=int, default=64)
    ex.add_argument("--k", type=int, default=8)
    ex.add_argument("--dim", type=int, default=7168)
    ex.add_argument("--hidden", type=int, default=2048)
    ex.add_argument("--repeat", type=int, default=3)
    ad = sub.add_parser("adapt")
    ad.add_argument("--requests", type=int, default=64)
    ad.add_argument("--length", type=int, default=1)
    ad.add_argument("--adapters", type=int, default=48)
    ad.add_argument("--rank", type=int, default=64)
    ad.add_argument("--dim", type=int, default=7168)
    ad.add_argument("--out-dim", type=int, default=8192)
    ad.add_argument("--repeat", type=int, default=3)
    args = ap.parse_args(argv)
    dev = torch.device("cuda", 0)
    torch.cuda.set_device(dev)

    if args.cmd == "prepare":
        M = args.tokens
        x, wq, wsf, pos = W.prefill_chain(M) if M == 4632 else W.decode_chain(M)
        lat = _bf16(x, dev)
        w, ws, p_ = torch.from_numpy(wq).to(dev), torch.from_numpy(wsf).to(dev), torch.from_numpy(pos).to(dev)
        q4 = torch.empty((M, iq.Q_DIM // 2), dtype=torch.uint8, device=dev)
        sf = torch.empty((M, iq.Q_DIM // 32), dtype=torch.uint8, device=dev)
        work = torch.empty(max(1, iq.prepare_q_workspace_bytes(M)), dtype=torch.uint8, device=dev)
        threshold = {"auto": None, "small": iq.SMALL_M_MAX, "pair": 0}[args.route]
        old = iq.set_small_m_threshold(threshold) if threshold is not None else None
        try:
            us = _time_calls(lambda: iq.prepare_q(lat, w, ws, p_, q_fp4=q4, q_sf=sf, workspace=work),
                             args.repeat, dev)
        finally:
            if old is not None:
                iq.set_small_m_threshold(old)
        print(f"prepare M={M} route={args.route}: " + " ".join(f"{u:.2f}" for u in us) + " us per call")
    elif args.cmd == "attend":
        _attend(args, dev)
    elif args.cmd == "experts":
        _experts(args, dev)
    elif args.cmd == "adapt":
        _adapt(args, dev)
    elif args.cmd == "indexer":
        M, N = args.queries, args.keys
        arrays = W.indexer_inputs(M, N, seed=1, causal=not args.full)
        q4, qs, k4, ks, w, L = (torch.from_numpy(a).to(dev) for a in arrays)
        logits = torch.empty((M, N), dtype=torch.float32, device=dev)
        idx = torch.empty((M, args.topk), dtype=torch.int32, device=dev)
        us_l = _time_calls(lambda: iq.indexer_logits(q4, qs, k4, ks, w, L, logits=logits), args.repeat, dev)
        us_t = _time_calls(lambda: iq.indexer_topk(logits, L, args.topk, indices=idx), args.repeat, dev)
        print(f"indexer {M}x{N} {'full' if args.full else 'causal'}: logits " + " ".join(f"{u:.2f}" for u in us_l)
              + f" us; top-{args.topk} " + " ".join(f"{u:.2f}" for u in us_t) + " us per call")
    else:
        xb = W.quant_blocks_input(args.rows, args.cols, seed=1)
        X = _bf16(xb, dev)
        Y = torch.empty((args.rows, args.cols), dtype=torch.uint8, device=dev)
        S = torch.empty((-(-args.cols // 512), (args.rows + 3) // 4 * 4), dtype=torch.int32, device=dev)
        us = _time_calls(lambda: iq.fp8_quant_1x128_ue8m0(X, y=Y, scales=S), args.repeat, dev)
        print(f"quant {args.rows}x{args.cols}: " + " ".join(f"{u:.2f}" for u in us) + " us per call")
    return 0 if iq.device_status() == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
