"""The operators of a scoring request with several samples, as cases that can be timed and compared.

A Prefill-Only request carries one prefix (instructions, user context) and several samples that
follow it; a request that draws several continuations has the same layout one token at a time.

  shared_prefill     attention of every sample token over its request's prefix and its own sample
                     up to itself (``bg_shared_prefill_attn``)
  shared_last_token  attention of one query per sample over the prefix and the whole sample
                     (``bg_shared_last_token_attn``): the last layer of a scoring request, or one
                     decode step of samples drawn from one prompt
  token_logprobs     log-probability of a given token, entropy and the best alternatives of rows of
                     logits (``bg_token_logprobs``)

``own`` chooses between the plain torch form and the library's kernels; both take what ``prepare``
makes and return the same tensors.
"""
import math
import random

import torch

own = False

PREFILL, LAST, LOGPROBS = "shared_prefill", "shared_last_token", "token_logprobs"


# --------------------------------------------------------------------------- cases
def _attn(name, op, requests, samples, prefix, own_len, hq, hkv, d, softcap=0.0, lengths=1):
    """``samples`` per request; prefix and sample lengths are uniform over their [lo, hi]."""
    return {"name": name, "op": op, "requests": requests, "samples": samples, "prefix_lo": prefix[0],
            "prefix_hi": prefix[1], "own_lo": own_len[0], "own_hi": own_len[1], "hq": hq, "hkv": hkv, "d": d,
            "softcap": softcap, "lengths": lengths}


def _rows(name, rows, vocab, dtype, top, masked):
    return {"name": name, "op": LOGPROBS, "rows": rows, "vocab": vocab, "dtype": dtype, "top": top, "masked": masked}


def listed():
    return [
        # one scoring request of 15 short samples, alone on the card: latency counts
        _attn("prefill_one_request", PREFILL, 1, 15, (400, 400), (16, 64), 16, 8, 128),
        # a batch of such requests, the ordinary load of a scoring service
        _attn("prefill_batch", PREFILL, 32, 15, (200, 500), (16, 96), 16, 8, 128),
        # the smaller model's heads (14 over 2, head_dim 64), capped scores, longer samples
        _attn("prefill_capped_d64", PREFILL, 16, 7, (1, 500), (1, 300), 14, 2, 64, softcap=30.0),
        # few requests that share a long document, samples of several hundred tokens: the largest prefill
        _attn("prefill_long_prefix", PREFILL, 2, 8, (8000, 8191), (257, 700), 16, 8, 128),
        # eight continuations of one long prompt: one decode step, alone on the card
        _attn("last_one_request", LAST, 1, 8, (4096, 4096), (1, 40), 16, 8, 128),
        # the last layer of prefill_batch's requests
        _attn("last_batch", LAST, 32, 15, (200, 500), (16, 96), 16, 8, 128),
        # capped scores, one kv head for seven query heads, odd lengths
        _attn("last_capped_d64", LAST, 24, 31, (333, 2047), (1, 77), 14, 2, 64, softcap=30.0),
        # decode over long shared prompts, continuations of up to 400 tokens: bound by reading K and V
        _attn("last_long_prefix", LAST, 4, 32, (30000, 32768), (1, 400), 32, 8, 128),
        # one next-token distribution, as after a single request
        _rows("logprobs_one_row", 1, 65536, "float32", 5, False),
        # the last tokens of a batch's samples, an odd vocabulary with banned tokens
        _rows("logprobs_samples", 480, 50001, "float32", 8, True),
        # every token of a long prompt scored, bf16 logits, the usual limit of alternatives
        _rows("logprobs_prompt", 8192, 65536, "bfloat16", 20, False),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is uniform over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice([PREFILL, PREFILL, LAST, LAST, LOGPROBS])
    if op == LOGPROBS:
        vocab = _log(rng, 1000, 160000)
        rows = _log(rng, 1, max(1, min(8192, 268435456 // vocab)))
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": rng.choice(["float32", "bfloat16"]),
                "top": rng.randint(1, 32), "masked": rng.random() < 0.5}
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
    while hq > 32:
        hq -= hkv
    requests = _log(rng, 1, 32)
    samples = _log(rng, 2, 32)
    # at most 16384 sample tokens; query x key pairs and prefix rows at most the largest listed cases'
    own_hi = _log(rng, 8, min(700, max(16, 16384 // (requests * samples))))
    most = 131072 // requests if op == LAST else 60000000 // (requests * samples * own_hi)
    prefix_hi = max(1, min(_log(rng, 16, 32768 if op == LAST else 8191), most))
    return {"op": op, "requests": requests, "samples": samples, "prefix_lo": rng.randint(0, prefix_hi),
            "prefix_hi": prefix_hi, "own_lo": rng.randint(1, own_hi), "own_hi": own_hi, "hq": hq, "hkv": hkv, "d": d,
            "softcap": rng.choice([0.0, 0.0, 30.0]), "lengths": rng.randint(0, 1 << 30)}


def _lengths(case):
    """(prefix lengths of the requests, sample lengths in packed order): the case's own, whatever the seed."""
    rng = random.Random(case["lengths"])
    prefix = [rng.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(case["requests"])]
    samples = [rng.randint(case["own_lo"], case["own_hi"]) for _ in range(case["requests"] * case["samples"])]
    return prefix, samples


# --------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    if case["op"] == LOGPROBS:
        rows, vocab = case["rows"], case["vocab"]
        # a language model's logits: a broad body and a few tokens well above it
        logits = torch.randn((rows, vocab), generator=gen, device="cuda") * 2.5
        peaks = torch.randint(vocab, (rows, 6), generator=gen, device="cuda")
        logits.scatter_add_(1, peaks, 4.0 + 2.0 * torch.randn((rows, 6), generator=gen, device="cuda"))
        tokens = torch.randint(vocab, (rows,), generator=gen, device="cuda")
        if case["masked"]:
            banned = torch.rand((vocab,), generator=gen, device="cuda") < 0.125
            given = logits.gather(1, tokens[:, None])
            logits.masked_fill_(banned, -math.inf)
            logits.scatter_(1, tokens[:, None], given)
        return {"op": LOGPROBS, "logits": logits.to(getattr(torch, case["dtype"])), "tokens": tokens.to(torch.int32),
                "top": case["top"]}

    prefix, samples = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    per = case["samples"]

    def offsets(lengths):
        cu = [0]
        for n in lengths:
            cu.append(cu[-1] + n)
        return torch.tensor(cu, dtype=torch.int32, device="cuda")

    total = sum(samples)
    rows = total if case["op"] == PREFILL else len(samples)
    q = normal(rows, hq, d)
    if case["softcap"]:
        q = q * 8          # scores that reach the cap
    return {"op": case["op"], "q": q, "k": normal(total, hkv, d), "v": normal(total, hkv, d),
            "prefix_k": normal(sum(prefix), hkv, d), "prefix_v": normal(sum(prefix), hkv, d),
            "cu_seqlens": offsets(samples), "max_seqlen": max(samples),
            "cu_prefix": offsets(prefix), "max_prefix_len": max(prefix),
            # samples cu_group[r] .. cu_group[r + 1] - 1 belong to request r
            "cu_group": torch.arange(case["requests"] + 1, dtype=torch.int32, device="cuda") * per,
            "max_group_tokens": max(sum(samples[r * per:(r + 1) * per]) for r in range(case["requests"])),
            "max_group_seqs": per, "scale": 1.0 / math.sqrt(d), "softcap": case["softcap"]}


# --------------------------------------------------------------------------- plain forms
def _plain_attn(s):
    """Each request as one padded row of a batch: its queries against [prefix ; its samples' keys]."""
    prefill = s["op"] == PREFILL
    q, cu, cup, cug = s["q"], s["cu_seqlens"].long(), s["cu_prefix"].long(), s["cu_group"].long()
    hq, d = q.shape[1], q.shape[2]
    hkv = s["k"].shape[1]
    R = cug.numel() - 1
    dev = q.device
    tok = cu[cug]                                            # first own token of each request, and the end
    plen, olen = cup[1:] - cup[:-1], tok[1:] - tok[:-1]
    P, M = s["max_prefix_len"], s["max_group_tokens"]

    def padded(x, start, n):                                 # [R, n, ...] fp32; rows past the end repeat the last
        at = (start[:, None] + torch.arange(n, device=dev)).clamp_(max=max(x.shape[0] - 1, 0))
        return x[at].float()

    keys, values = padded(s["k"], tok[:-1], M), padded(s["v"], tok[:-1], M)
    if P:
        keys = torch.cat((padded(s["prefix_k"], cup[:-1], P), keys), 1)
        values = torch.cat((padded(s["prefix_v"], cup[:-1], P), values), 1)
    # the rows of a request, and the packed keys that each sees: its sample's start up to itself, or to its end
    first, n = (tok, M) if prefill else (cug, s["max_group_seqs"])
    row = first[:-1, None] + torch.arange(n, device=dev)
    live = row < first[1:, None]
    row = row.clamp(max=q.shape[0] - 1)
    if prefill:
        lo, hi = cu[torch.searchsorted(cu, row, right=True) - 1], row + 1
    else:
        lo, hi = cu[row], cu[row + 1]
    at = tok[:-1, None] + torch.arange(M, device=dev)
    sees = (at[:, None, :] >= lo[:, :, None]) & (at[:, None, :] < hi[:, :, None])
    if P:
        sees = torch.cat(((torch.arange(P, device=dev) < plen[:, None])[:, None, :].expand(R, n, P), sees), 2)

    qp = q[row].float().view(R, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)              # [R, hkv, g, n, d]
    x = torch.matmul(qp, keys.permute(0, 2, 3, 1)[:, :, None]) * s["scale"]
    if s["softcap"]:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    x = x.masked_fill(~sees[:, None, None], -math.inf)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(w / w.sum(-1, keepdim=True), values.permute(0, 2, 1, 3)[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(R, n, hq, d)
    return o[live].to(q.dtype)                               # rows in packed order


def _plain_logprobs(s):
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    z = e.sum(-1, keepdim=True)
    lse = top + torch.log(z)
    p = e / z
    entropy = torch.where(p > 0, p * (lse - x), torch.zeros_like(p)).sum(-1)
    logprob = (x.gather(1, s["tokens"].long()[:, None]) - lse)[:, 0]
    best, at = torch.sort(x, dim=-1, descending=True, stable=True)    # ties: the lowest token first
    k = s["top"]
    return {"logprob": logprob, "entropy": entropy, "top_token": at[:, :k].to(torch.int32),
            "top_logprob": best[:, :k] - lse}


# --------------------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return _plain_logprobs(s) if s["op"] == LOGPROBS else _plain_attn(s)
    from attention_packed_varlen_causal_gb300 import binding as bg
    if s["op"] == LOGPROBS:
        rows, k = s["logits"].shape[0], s["top"]
        f32 = {"dtype": torch.float32, "device": s["logits"].device}
        out = {"logprob": torch.empty(rows, **f32), "entropy": torch.empty(rows, **f32),
               "top_token": torch.empty((rows, k), dtype=torch.int32, device=f32["device"]),
               "top_logprob": torch.empty((rows, k), **f32)}
        bg.bg_token_logprobs(s["logits"], s["tokens"], **out)
        return out
    if "workspace" not in s:                                 # kept by the caller, as for the other attention calls
        size = bg.bg_shared_attn_workspace_size(
            s["cu_group"].numel() - 1, s["cu_seqlens"].numel() - 1, s["k"].shape[0], s["max_seqlen"],
            s["max_prefix_len"], s["q"].shape[1], s["k"].shape[1], s["q"].shape[2])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["q"].device)
    call = bg.bg_shared_prefill_attn if s["op"] == PREFILL else bg.bg_shared_last_token_attn
    out = torch.empty_like(s["q"])
    call(s["q"], s["k"], s["v"], s["cu_seqlens"], s["max_seqlen"], s["prefix_k"], s["prefix_v"], s["cu_prefix"],
         s["max_prefix_len"], s["cu_group"], out, scale=s["scale"], softcap=s["softcap"], workspace=s["workspace"])
    return out


# --------------------------------------------------------------------------- work
def work(case):
    """Each input read once and each output written once; two multiply-adds of head_dim per visible pair."""
    if case["op"] == LOGPROBS:
        n = case["rows"] * case["vocab"]
        # per logit: the difference, the exponential, its sum and the entropy's multiply-add
        return {"bytes": n * (4 if case["dtype"] == "float32" else 2) + case["rows"] * (4 + 8 + 8 * case["top"]),
                "flops": 5 * n}
    prefix, samples = _lengths(case)
    hq, hkv, d, per = case["hq"], case["hkv"], case["d"], case["samples"]
    pairs = 0
    for i, n in enumerate(samples):
        p = prefix[i // per]
        pairs += n * p + n * (n + 1) // 2 if case["op"] == PREFILL else p + n
    rows = sum(samples) if case["op"] == PREFILL else len(samples)
    return {"bytes": 2 * d * (2 * rows * hq + 2 * hkv * (sum(samples) + sum(prefix))), "flops": 4 * d * hq * pairs}


# --------------------------------------------------------------------------- definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == LOGPROBS:
        if case["rows"] * case["vocab"] > 1 << 30:
            return None
        outs = []
        for part, given in zip(s["logits"].split(256), s["tokens"].split(256)):     # rows are independent
            x = part.double()
            logp = x - torch.logsumexp(x, -1, keepdim=True)
            # the first `top` columns by value, the lower index first among equals: a stable sort's
            order = torch.argsort(-x, dim=-1, stable=True)[:, :case["top"]]
            outs.append((logp.gather(1, given.long()[:, None])[:, 0],
                         torch.special.entr(logp.exp()).sum(-1), order.to(torch.int32), logp.gather(1, order)))
        cat = [torch.cat(t) for t in zip(*outs)]
        return dict(zip(("logprob", "entropy", "top_token", "top_logprob"), cat))
    prefix, samples = _lengths(case)
    g, cap = case["hq"] // case["hkv"], case["softcap"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    at = p0 = 0
    for i, n in enumerate(samples):                          # one sample at a time over [prefix ; sample]
        r = i // case["samples"]
        if i and i % case["samples"] == 0:
            p0 += prefix[r - 1]
        k = torch.cat((s["prefix_k"][p0:p0 + prefix[r]], s["k"][at:at + n])).double().repeat_interleave(g, 1)
        v = torch.cat((s["prefix_v"][p0:p0 + prefix[r]], s["v"][at:at + n])).double().repeat_interleave(g, 1)
        rows = slice(at, at + n) if case["op"] == PREFILL else slice(i, i + 1)
        x = torch.einsum("qhd,khd->hqk", s["q"][rows].double(), k) * s["scale"]
        if cap:
            x = cap * torch.tanh(x / cap)
        if case["op"] == PREFILL:
            later = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
            x[:, :, prefix[r]:].masked_fill_(later, -math.inf)
        out[rows] = torch.einsum("hqk,khd->qhd", torch.softmax(x, -1), v)
        at += n
    return out
