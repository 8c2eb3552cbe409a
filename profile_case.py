"""Runs one hot-path call on a named workload a few times, for profilers.

    python profile_case.py prefill_only --iters 3
    python profile_case.py beam_long --iters 2
    python profile_case.py beam_long --iters 2 --two-call
    python profile_case.py select_long --iters 2
    python profile_case.py prefill_only --iters 3 --fp8
    python profile_case.py shared_prefill --iters 3
    python profile_case.py shared_last --iters 3
    python profile_case.py logprobs --iters 3
    python profile_case.py rope --iters 3
    python profile_case.py adjust --iters 3
    python profile_case.py tree --iters 3

Prefill workloads (tiny, prefill_only, skewed) call bg_packed_prefill_attn
``iters`` times on one layer of inputs; decode workloads (beam_short,
beam_long) run ``iters`` complete beam searches of one layer (per step the
suffix reorder + append, then the decode attention: one bg_beam_decode_step
call, or with ``--two-call`` bg_beam_suffix_reorder, then
bg_beam_decode_attn); selection workloads
(select_short, select_long) call bg_beam_select ``iters`` times on the beam
configurations' shapes with fp32 logits N(0, 3) over 65,536 tokens;
shared_prefill and shared_last call bg_shared_prefill_attn and
bg_shared_last_token_attn on 32 requests of 15 samples of 56 tokens after a
prefix of 350 (16/8 heads, d 128); logprobs calls bg_token_logprobs on 8192 rows of
65,536 bf16 logits; rope calls bg_packed_qk_norm_rope on prefill_only's tokens out of
a fused projection; adjust calls bg_adjust_logits on 8 searches of 100 beams over
65,536 fp32 logits, prompts of 500 tokens, 2% of the tokens allowed; tree calls
bg_tree_attn on 8 drafts of 52 nodes over 8,000 keys (32/8 heads, d 128).  Inputs are drawn on the device with a seeded generator,
shaped as in ``workloads``.  Nothing is
timed here: use ncu (or bench.py for timings).
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def main(argv=None):
    import numpy as np
    import torch

    from attention_packed_varlen_causal_gb300 import binding as bg
    from attention_packed_varlen_causal_gb300 import build
    from attention_packed_varlen_causal_gb300 import workloads as wl

    ap = argparse.ArgumentParser()
    select = {"select_short": "beam_short", "select_long": "beam_long"}
    scoring = ["shared_prefill", "shared_last", "logprobs"]
    steps = ["rope", "adjust", "tree"]
    ap.add_argument("workload", choices=sorted(list(wl.PREFILL_CONFIGS) + list(wl.DECODE_CONFIGS) + list(select) + scoring + steps))
    ap.add_argument("--iters", type=int, default=3)
    ap.add_argument("--two-call", action="store_true", help="decode: separate reorder and attention calls")
    ap.add_argument("--fp8", action="store_true", help="prefill: E4M3 Q and K (bg_packed_prefill_attn_fp8)")
    args = ap.parse_args(argv)
    build.build()
    bg.load()
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(1234)
    bf = torch.bfloat16
    if args.workload in select:
        cfg = wl.DECODE_CONFIGS[select[args.workload]]
        R, W, V = cfg.R, cfg.W, 65536
        logits = torch.randn((R, W, V), generator=g, device=dev) * 3.0
        cum = torch.randn((R, W), generator=g, device=dev) - 3.0
        tok = torch.empty((R, W), dtype=torch.int32, device=dev)
        par = torch.empty_like(tok)
        sc = torch.empty((R, W), dtype=torch.float32, device=dev)
        ws = torch.empty(bg.bg_beam_select_workspace_size(R, W, V), dtype=torch.uint8, device=dev)
        for _ in range(args.iters):
            bg.bg_beam_select(logits, cum, tok, par, sc, workspace=ws)
    elif args.workload == "logprobs":
        N, V, K = 8192, 65536, 20
        logits = (torch.randn((N, V), generator=g, device=dev) * 3.0).to(bf)
        tok = torch.randint(V, (N,), generator=g, device=dev, dtype=torch.int32)
        lp, ent = (torch.empty(N, dtype=torch.float32, device=dev) for _ in range(2))
        tt = torch.empty((N, K), dtype=torch.int32, device=dev)
        tl = torch.empty((N, K), dtype=torch.float32, device=dev)
        for _ in range(args.iters):
            bg.bg_token_logprobs(logits, tok, logprob=lp, entropy=ent, top_token=tt, top_logprob=tl)
    elif args.workload == "rope":
        cfg = wl.PREFILL_CONFIGS["prefill_only"]
        T, Hq, Hkv, d = sum(wl.prefill_lengths(cfg)), cfg.Hq, cfg.Hkv, cfg.head_dim
        x = torch.randn((T, (Hq + 2 * Hkv) * d), generator=g, device=dev).to(bf)
        q, k, v = (t.unflatten(-1, (-1, d)) for t in x.split((Hq * d, Hkv * d, Hkv * d), -1))
        pos = torch.randint(cfg.hi, (T,), generator=g, device=dev, dtype=torch.int32)
        w = torch.ones(d, dtype=bf, device=dev)
        f = (1e6 ** (-torch.arange(d // 2, device=dev) * 2 / d)).float()
        out = [torch.empty((T, h, d), dtype=bf, device=dev) for h in (Hq, Hkv, Hkv)]
        for _ in range(args.iters):
            bg.bg_packed_qk_norm_rope(q, k, v, pos, *out, inv_freq=f, q_weight=w, k_weight=w)
    elif args.workload == "adjust":
        G, W, V, P, M = 8, 100, 65536, 500, 512
        x = torch.randn((G * W, V), generator=g, device=dev) * 2.5
        out = torch.empty_like(x)

        def tokens(*shape):
            return (torch.rand(shape, generator=g, device=dev) ** 3 * V).to(torch.int32)

        bits = torch.rand((M, V // 32, 32), generator=g, device=dev) < 0.02
        mask = (bits.long() << torch.arange(32, device=dev)).sum(-1).to(torch.uint32).view(torch.int32)
        kw = dict(rows_per_group=W, prompt_tokens=tokens(G * P), cu_prompt=torch.arange(G + 1, dtype=torch.int32, device=dev) * P,
                  own_tokens=tokens(G * W, 4), repetition=torch.full((G,), 1.2, device=dev), mask=mask,
                  mask_index=torch.randint(M, (G * W,), generator=g, device=dev, dtype=torch.int32))
        for _ in range(args.iters):
            bg.bg_adjust_logits(x, out, **kw)
    elif args.workload == "tree":
        R, n, plen, Hq, Hkv, d = 8, 52, 8000, 32, 8, 128
        q = torch.randn((R * n, Hq, d), generator=g, device=dev).to(bf)
        k, v = (torch.randn((R * n, Hkv, d), generator=g, device=dev).to(bf) for _ in range(2))
        pk, pv = (torch.randn((R * plen, Hkv, d), generator=g, device=dev).to(bf) for _ in range(2))
        parent = torch.arange(R * n, dtype=torch.int32, device=dev) % n // 2 - 1
        cu = torch.arange(R + 1, dtype=torch.int32, device=dev) * n
        cup = torch.arange(R + 1, dtype=torch.int32, device=dev) * plen
        out = torch.empty_like(q)
        ws = torch.empty(bg.bg_tree_attn_workspace_size(R, R * n, n, plen, Hq, Hkv, d), dtype=torch.uint8, device=dev)
        for _ in range(args.iters):
            bg.bg_tree_attn(q, k, v, parent, cu, n, pk, pv, cup, plen, out, workspace=ws)
    elif args.workload in scoring:
        R, S, n, plen, Hq, Hkv, d = 32, 15, 56, 350, 16, 8, 128
        last = args.workload == "shared_last"
        T = R * S * n
        q = torch.randn((R * S if last else T, Hq, d), generator=g, device=dev).to(bf)
        k, v = (torch.randn((T, Hkv, d), generator=g, device=dev).to(bf) for _ in range(2))
        pk, pv = (torch.randn((R * plen, Hkv, d), generator=g, device=dev).to(bf) for _ in range(2))
        cu = torch.arange(R * S + 1, dtype=torch.int32, device=dev) * n
        cup = torch.arange(R + 1, dtype=torch.int32, device=dev) * plen
        cug = torch.arange(R + 1, dtype=torch.int32, device=dev) * S
        out = torch.empty_like(q)
        ws = torch.empty(bg.bg_shared_attn_workspace_size(R, R * S, T, n, plen, Hq, Hkv, d), dtype=torch.uint8, device=dev)
        call = bg.bg_shared_last_token_attn if last else bg.bg_shared_prefill_attn
        for _ in range(args.iters):
            call(q, k, v, cu, n, pk, pv, cup, plen, cug, out, workspace=ws)
    elif args.workload in wl.PREFILL_CONFIGS:
        cfg = wl.PREFILL_CONFIGS[args.workload]
        lengths = wl.prefill_lengths(cfg)
        cu_np = wl.cu_from_lengths(lengths)
        T = int(cu_np[-1])
        q = torch.randn((T, cfg.Hq, cfg.head_dim), generator=g, device=dev).to(bf)
        k = torch.randn((T, cfg.Hkv, cfg.head_dim), generator=g, device=dev).to(bf)
        v = torch.randn((T, cfg.Hkv, cfg.head_dim), generator=g, device=dev).to(bf)
        out = torch.empty_like(q)
        cu = torch.from_numpy(cu_np).to(dev)
        ws = torch.empty(bg.bg_packed_prefill_workspace_size(len(lengths), T, max(lengths), cfg.Hq, cfg.Hkv,
                                                             cfg.head_dim), dtype=torch.uint8, device=dev)
        if args.fp8:
            # E4M3 codes of q and k with one power-of-two scale each (max |x| / scale <= 448)
            codes = []
            for x in (q, k):
                s8 = 2.0 ** math.ceil(math.log2(float(x.abs().max().float().item()) / 448.0))
                codes.append(((x.float() / s8).to(torch.float8_e4m3fn).view(torch.uint8), s8))
            for _ in range(args.iters):
                bg.bg_packed_prefill_attn_fp8(codes[0][0], codes[0][1], codes[1][0], codes[1][1], v, cu, max(lengths),
                                              out, workspace=ws)
        else:
            for _ in range(args.iters):
                bg.bg_packed_prefill_attn(q, k, v, cu, max(lengths), out, workspace=ws)
    else:
        cfg = wl.DECODE_CONFIGS[args.workload]
        plen = wl.decode_prompt_lengths(cfg)
        cu_np = wl.cu_from_lengths(plen)
        P = int(cu_np[-1])
        R, W, Hq, Hkv, d, S = cfg.R, cfg.W, cfg.Hq, cfg.Hkv, cfg.head_dim, cfg.steps
        pk = torch.randn((P, Hkv, d), generator=g, device=dev).to(bf)
        pv = torch.randn((P, Hkv, d), generator=g, device=dev).to(bf)
        cu = torch.from_numpy(cu_np).to(dev)
        qs = [torch.randn((R, W, Hq, d), generator=g, device=dev).to(bf) for _ in range(S)]
        nk = [torch.randn((R, W, Hkv, d), generator=g, device=dev).to(bf) for _ in range(S)]
        nv = [torch.randn((R, W, Hkv, d), generator=g, device=dev).to(bf) for _ in range(S)]
        parents = [torch.from_numpy(np.random.default_rng(wl.SEED_PARENT + s).integers(0, W, size=(R, W))
                                    .astype(np.int32)).to(dev) for s in range(S)]
        sk = [torch.zeros((R, W, S, Hkv, d), dtype=bf, device=dev) for _ in range(2)]
        sv = [torch.zeros((R, W, S, Hkv, d), dtype=bf, device=dev) for _ in range(2)]
        out = torch.empty_like(qs[0])
        for _ in range(args.iters):
            for s in range(S):
                src, dst = s % 2, 1 - s % 2
                if not args.two_call:
                    bg.bg_beam_decode_step(qs[s], pk, pv, cu, max(plen), sk[src], sv[src], parents[s], nk[s], nv[s],
                                           sk[dst], sv[dst], s + 1, out)
                    continue
                bg.bg_beam_suffix_reorder(sk[src], sv[src], sk[dst], sv[dst], parents[s], s, new_k=nk[s],
                                          new_v=nv[s])
                bg.bg_beam_decode_attn(qs[s], pk, pv, cu, max(plen), sk[dst], sv[dst], s + 1, out)
    torch.cuda.synchronize()
    print(f"profile_case {args.workload}: {args.iters} iteration(s) done")


if __name__ == "__main__":
    main()
