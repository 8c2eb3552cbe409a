"""The operators around the attention of a decode or verify step, as cases that can be timed and compared.

  rope        norm of every head of q and k and the rotation by the token's position, out of the fused
              projection's rows into the tensors that the packed prefill reads (``bg_packed_qk_norm_rope``);
              positions with several axes for images and video
  beam_rope   the same for the one new token of every beam of a search, K and V straight into the beams'
              suffix (``bg_beam_qk_norm_rope``)
  logits      penalties for repeated tokens, biases and grammar masks on rows of logits, ahead of the
              candidate selection or the sampling (``bg_adjust_logits``)
  tree        attention of a tree of drafted tokens over a request's cached prefix and each token's own
              ancestors (``bg_tree_attn``)

``own`` chooses between the plain torch form and the library's kernels; both take what ``prepare`` makes
and return the same tensors.
"""
import math
import random

import torch

own = False

ROPE, BEAM, LOGITS, TREE = "rope", "beam_rope", "logits", "tree"


# --------------------------------------------------------------------------- cases
def _rope(name, tokens, hq, hkv, d, axes=1, rot=None, norm=True, interleaved=False, longest=500):
    """``rot``: rotated dimensions of a head; ``longest``: positions are below it."""
    return {"name": name, "op": ROPE, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "axes": axes,
            "rot": d if rot is None else rot, "norm": norm, "interleaved": interleaved, "longest": longest}


def _beam(name, requests, width, hq, hkv, d, step, slots, prompt):
    return {"name": name, "op": BEAM, "requests": requests, "width": width, "hq": hq, "hkv": hkv, "d": d, "axes": 1,
            "rot": d, "norm": True, "interleaved": False, "step": step, "slots": slots, "longest": prompt}


def _logits(name, groups, per, vocab, dtype, prompt, own_len, bias, masks, allowed):
    """``per`` rows share a prompt of up to ``prompt`` tokens and ``bias`` biased tokens, each has up to
    ``own_len`` tokens of its own; ``masks`` grammar states that allow a share of the vocabulary."""
    return {"name": name, "op": LOGITS, "groups": groups, "per": per, "vocab": vocab, "dtype": dtype, "prompt": prompt,
            "own_len": own_len, "bias": bias, "masks": masks, "allowed": allowed}


def _tree(name, requests, nodes, prefix, hq, hkv, d, softcap=0.0, lengths=1):
    """Nodes and prefix lengths are uniform over their [lo, hi]."""
    return {"name": name, "op": TREE, "requests": requests, "nodes_lo": nodes[0], "nodes_hi": nodes[1],
            "prefix_lo": prefix[0], "prefix_hi": prefix[1], "hq": hq, "hkv": hkv, "d": d, "softcap": softcap,
            "lengths": lengths}


def listed():
    return [
        # one small packed batch: latency counts
        _rope("rope_one_batch", 392, 16, 8, 128, longest=211),
        # a layer of a full Prefill-Only batch (240 sequences)
        _rope("rope_prefill", 70375, 16, 8, 128),
        # the smaller model's heads, images and video among the text: time, height and width
        _rope("rope_images_d64", 23041, 14, 2, 64, axes=3, longest=4000),
        # a long document, half of each head rotated, neighbouring pairs, no norm
        _rope("rope_partial", 32768, 32, 8, 128, rot=64, norm=False, interleaved=True, longest=32768),
        # the new tokens of one request's beams: latency counts
        _beam("beam_rope_one", 1, 100, 16, 8, 128, 2, 5, 400),
        # a decode step of a search of 400 beams, the smaller model's heads
        _beam("beam_rope_long", 16, 400, 14, 2, 64, 4, 5, 500),
        # one next-token distribution of a request that draws one answer
        _logits("logits_one_row", 1, 1, 65536, "float32", 500, 40, 16, 0, 0.0),
        # a step of 32 searches of 100 beams whose tokens are identifiers from a tree: few tokens allowed
        _logits("logits_beams", 32, 100, 65536, "float32", 500, 4, 8, 512, 0.02),
        # answers with long histories of their own, an odd vocabulary, bf16 logits, a lax grammar
        _logits("logits_samples", 32, 15, 50001, "bfloat16", 4000, 700, 300, 64, 0.6),
        # one request's draft verified over its prompt: latency counts
        _tree("tree_one_request", 1, (26, 26), (4096, 4096), 16, 8, 128),
        # a batch of requests with short prompts, capped scores, seven query heads to a kv head
        _tree("tree_batch_capped_d64", 32, (8, 63), (200, 2047), 14, 2, 64, softcap=30.0),
        # large drafts over long documents: bound by reading K and V
        _tree("tree_long_prefix", 8, (40, 64), (30000, 32768), 32, 8, 128),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is uniform over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _heads(rng):
    hkv = rng.choice([1, 2, 3, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 7])
    return (hq if hq <= 32 else 4 * hkv), hkv, rng.choice([64, 128])


def draw(rng):
    op = rng.choice([ROPE, ROPE, BEAM, LOGITS, LOGITS, TREE, TREE, TREE])
    hq, hkv, d = _heads(rng)
    if op == LOGITS:
        vocab = _log(rng, 1000, 160000)
        rows = _log(rng, 1, max(1, min(3200, 209715200 // vocab)))
        groups = _log(rng, 1, rows)
        masks = rng.choice([0, _log(rng, 1, 512)])
        return {"op": op, "groups": groups, "per": max(1, rows // groups), "vocab": vocab,
                "dtype": rng.choice(["float32", "bfloat16"]), "prompt": _log(rng, 1, 8000), "own_len": _log(rng, 1, 1000),
                "bias": rng.choice([0, _log(rng, 1, 300)]), "masks": masks, "allowed": rng.choice([0.001, 0.02, 0.3, 0.9])}
    if op == TREE:
        requests = _log(rng, 1, 32)
        nodes_hi = _log(rng, 2, min(256, 4096 // requests))
        prefix_hi = min(_log(rng, 16, 32768), 262144 // requests, 16777216 // (requests * nodes_hi))
        return {"op": op, "requests": requests, "nodes_lo": rng.randint(1, nodes_hi), "nodes_hi": nodes_hi,
                "prefix_lo": rng.randint(0, prefix_hi), "prefix_hi": prefix_hi, "hq": hq, "hkv": hkv, "d": d,
                "softcap": rng.choice([0.0, 0.0, 30.0]), "lengths": rng.randint(0, 1 << 30)}
    axes = rng.choice([1, 1, 2, 3])
    case = {"op": op, "hq": hq, "hkv": hkv, "d": d, "axes": axes, "rot": rng.choice([d, d, d // 2, d - 16]),
            "norm": rng.random() < 0.75, "interleaved": rng.random() < 0.25, "longest": _log(rng, 100, 131072)}
    if op == ROPE:
        return dict(case, tokens=_log(rng, 1, 288000000 // ((hq + 2 * hkv) * d)))
    slots = rng.randint(1, 16)
    return dict(case, requests=_log(rng, 1, 32), width=rng.randint(1, 400), step=rng.randint(0, 15), slots=slots)


def _lengths(case):
    """(nodes, prefix length) of each request of a tree case: the case's own, whatever the seed."""
    rng = random.Random(case["lengths"])
    nodes = [rng.randint(case["nodes_lo"], case["nodes_hi"]) for _ in range(case["requests"])]
    prefix = [rng.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(case["requests"])]
    return nodes, prefix


# --------------------------------------------------------------------------- inputs
def _offsets(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _parents(rng, n):
    """A draft: some candidates for the next token, most of the later ones below a recent one."""
    return [rng.randint(-1, min(i - 1, 3)) if rng.random() < 0.3 else rng.randint(max(-1, i - 6), i - 1) for i in range(n)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)

    op = case["op"]
    if op in (ROPE, BEAM):
        hq, hkv, d, axes, half = case["hq"], case["hkv"], case["d"], case["axes"], case["rot"] // 2
        rows = case["tokens"] if op == ROPE else case["requests"] * case["width"]
        at = torch.arange(half, device="cuda", dtype=torch.float64)
        s = {"op": op, "hq": hq, "hkv": hkv, "d": d, "qkv": normal(rows, (hq + 2 * hkv) * d), "eps": 1e-6,
             "inv_freq": (1e6 ** (-at / half)).float(), "interleaved": case["interleaved"],
             "q_weight": (1 + 0.2 * normal(d, dtype=torch.float32)).bfloat16() if case["norm"] else None,
             "k_weight": (1 + 0.2 * normal(d, dtype=torch.float32)).bfloat16() if case["norm"] else None,
             # sections of the frequencies for time, height and width: a quarter, and the rest in equal parts
             "axis_of": None if axes == 1 else [0 if 4 * i < half else 1 + (4 * i - half) * (axes - 1) // (3 * half)
                                                for i in range(half)]}
        if op == ROPE:
            s["positions"] = whole(0, case["longest"], axes, rows)
            return s
        s.update(requests=case["requests"], width=case["width"], step=case["step"], slot=min(case["step"], case["slots"] - 1),
                 base_pos=whole(1, case["longest"] + 1, axes, case["requests"]))
        shape = (case["requests"], case["width"], case["slots"], hkv, d)
        s.update(suffix_k=normal(*shape), suffix_v=normal(*shape))
        return s

    if op == LOGITS:
        groups, per, vocab = case["groups"], case["per"], case["vocab"]
        rows, rng = groups * per, random.Random(seed)
        logits = torch.randn((rows, vocab), generator=gen, device="cuda") * 2.5
        prompt = [rng.randint((case["prompt"] + 1) // 2, case["prompt"]) for _ in range(groups)]
        words = (vocab + 31) // 32
        # text repeats itself: tokens are frequent ones more often than not
        def text(*shape):
            u = torch.rand(shape, generator=gen, device="cuda")
            return (u * u * u * vocab).to(torch.int32).clamp_(max=vocab - 1)

        s = {"op": op, "logits": logits.to(getattr(torch, case["dtype"])), "per": per,
             "prompt_tokens": text(sum(prompt)), "cu_prompt": _offsets(prompt), "own_tokens": text(rows, case["own_len"]),
             "own_lens": whole((case["own_len"] + 1) // 2, case["own_len"] + 1, rows),
             "repetition": 1.0 + 0.3 * torch.rand((groups,), generator=gen, device="cuda"),
             "frequency": 0.5 * torch.rand((groups,), generator=gen, device="cuda"),
             "presence": torch.rand((groups,), generator=gen, device="cuda") - 0.25,
             "bias_tokens": None, "bias_values": None, "cu_bias": None, "mask": None, "mask_index": None}
        if case["bias"]:
            n = case["bias"]
            # without repetition within a group: n places of a stride that visits all of them
            first, stride = whole(0, vocab, groups, 1).long(), vocab // max(n, 1)
            s["bias_tokens"] = ((first + torch.arange(n, device="cuda") * max(stride, 1)) % vocab).to(torch.int32).reshape(-1)
            s["bias_values"] = 3.0 * normal(groups * n, dtype=torch.float32)
            s["cu_bias"] = torch.arange(groups + 1, dtype=torch.int32, device="cuda") * n
        if case["masks"]:
            bits = torch.rand((case["masks"], words, 32), generator=gen, device="cuda") < case["allowed"]
            value = (bits.long() << torch.arange(32, device="cuda")).sum(-1)
            s["mask"] = torch.where(value >= 1 << 31, value - (1 << 32), value).to(torch.int32)
            # the grammar state of each row; a few are free of any
            s["mask_index"] = whole(0, case["masks"], rows)
            s["mask_index"][whole(0, rows, max(1, rows // 32)).long()] = -1
        return s

    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    nodes, prefix = _lengths(case)
    rng = random.Random(seed)
    total = sum(nodes)
    q = normal(total, hq, d)
    return {"op": op, "q": q * 8 if case["softcap"] else q,       # scores that reach the cap
            "k": normal(total, hkv, d), "v": normal(total, hkv, d),
            "prefix_k": normal(sum(prefix), hkv, d), "prefix_v": normal(sum(prefix), hkv, d),
            "parent": torch.tensor([p for n in nodes for p in _parents(rng, n)], dtype=torch.int32, device="cuda"),
            "cu_nodes": _offsets(nodes), "max_nodes": max(nodes), "cu_prefix": _offsets(prefix),
            "max_prefix_len": max(prefix), "scale": 1.0 / math.sqrt(d), "softcap": case["softcap"]}


# --------------------------------------------------------------------------- plain forms
def _normed(x, weight, eps):
    x = x.float()
    if weight is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()


def _rotated(x, angle, interleaved):
    """x [rows, heads, d] in fp32, angle [rows, rot / 2] in fp64: pairs (2 i, 2 i + 1) or (i, i + rot / 2)."""
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half = angle.shape[-1]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, rest), -1)


def _split(s):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    q, k, v = s["qkv"].split((hq * d, hkv * d, hkv * d), -1)
    return q.unflatten(-1, (hq, d)), k.unflatten(-1, (hkv, d)), v.unflatten(-1, (hkv, d))


def _plain_rope(s):
    q, k, v = _split(s)
    if s["op"] == ROPE:
        pos = s["positions"]
    else:
        pos = (s["base_pos"] + s["step"]).repeat_interleave(s["width"], 1)
    pos = pos.double()
    by_axis = pos[0][:, None] if s["axis_of"] is None else pos[torch.tensor(s["axis_of"], device=pos.device)].T
    angle = by_axis * s["inv_freq"].double()
    q = _rotated(_normed(q, s["q_weight"], s["eps"]), angle, s["interleaved"]).to(s["qkv"].dtype)
    k = _rotated(_normed(k, s["k_weight"], s["eps"]), angle, s["interleaved"]).to(s["qkv"].dtype)
    if s["op"] == ROPE:
        return {"q": q, "k": k, "v": v.contiguous()}
    rw = (s["requests"], s["width"])
    s["suffix_k"][:, :, s["slot"]] = k.unflatten(0, rw)
    s["suffix_v"][:, :, s["slot"]] = v.unflatten(0, rw)
    return {"q": q.unflatten(0, rw), "k": s["suffix_k"], "v": s["suffix_v"]}


def _plain_logits(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    per, dev = s["per"], x.device
    groups = rows // per
    group = torch.arange(rows, device=dev) // per
    cu = s["cu_prompt"].long()
    owner = torch.searchsorted(cu, torch.arange(s["prompt_tokens"].numel(), device=dev), right=True) - 1
    in_prompt = torch.zeros((groups, vocab), dtype=torch.bool, device=dev)
    in_prompt[owner, s["prompt_tokens"].long()] = True
    live = torch.arange(s["own_tokens"].shape[1], device=dev) < s["own_lens"][:, None]
    count = torch.zeros_like(x).scatter_add_(1, s["own_tokens"].long(), live.float())
    rep = s["repetition"][group][:, None]
    y = torch.where(in_prompt[group] | (count > 0), torch.where(x > 0, x / rep, x * rep), x)
    y = y - (s["frequency"][group][:, None] * count + s["presence"][group][:, None] * (count > 0))
    if s["bias_tokens"] is not None:
        bias = torch.zeros((groups, vocab), device=dev)
        bias.scatter_(1, s["bias_tokens"].long().view(groups, -1), s["bias_values"].view(groups, -1))
        y = y + bias[group]
    if s["mask"] is not None:
        at = torch.arange(vocab, device=dev)
        allowed = (s["mask"][:, at // 32] >> (at % 32).to(torch.int32)) & 1 == 1
        free = s["mask_index"] < 0
        y = y.masked_fill(~(allowed[s["mask_index"].clamp(min=0).long()] | free[:, None]), -math.inf)
    return y


def _plain_tree(s):
    """Each request as one padded row of a batch: its nodes against [prefix ; nodes]."""
    q, cun, cup = s["q"], s["cu_nodes"].long(), s["cu_prefix"].long()
    total, hq, d = q.shape
    hkv, dev = s["k"].shape[1], q.device
    R, M, P = cun.numel() - 1, s["max_nodes"], s["max_prefix_len"]

    def rows_of(cu, n):
        at = cu[:-1, None] + torch.arange(n, device=dev)
        return at, at < cu[1:, None]

    at, live = rows_of(cun, M)
    at = at.clamp(max=total - 1)
    # ancestors: the sum of all powers of the parents' matrix, which is strictly lower triangular
    parent = s["parent"].long()[at].masked_fill(~live, -1)
    up = (torch.arange(M, device=dev) == parent[..., None]).double()
    eye = torch.eye(M, device=dev, dtype=torch.float64).expand(R, M, M)
    sees = torch.linalg.solve_triangular(eye - up, eye, upper=False, unitriangular=True) > 0.5
    keys, values = s["k"][at].float(), s["v"][at].float()
    if P:
        pat, plive = rows_of(cup, P)
        pat = pat.clamp(max=s["prefix_k"].shape[0] - 1)
        keys = torch.cat((s["prefix_k"][pat].float(), keys), 1)
        values = torch.cat((s["prefix_v"][pat].float(), values), 1)
        sees = torch.cat((plive[:, None, :].expand(R, M, P), sees), 2)
    qp = q[at].float().view(R, M, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)              # [R, hkv, g, M, d]
    x = torch.matmul(qp, keys.permute(0, 2, 3, 1)[:, :, None]) * s["scale"]
    if s["softcap"]:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    x = x.masked_fill(~sees[:, None, None], -math.inf)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(w / w.sum(-1, keepdim=True), values.permute(0, 2, 1, 3)[:, :, None])
    return o.permute(0, 3, 1, 2, 4).reshape(R, M, hq, d)[live].to(q.dtype)


# --------------------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return {ROPE: _plain_rope, BEAM: _plain_rope, LOGITS: _plain_logits, TREE: _plain_tree}[s["op"]](s)
    from attention_packed_varlen_causal_gb300 import binding as bg
    op = s["op"]
    if op == LOGITS:
        out = torch.empty(s["logits"].shape, dtype=torch.float32, device=s["logits"].device)
        bg.bg_adjust_logits(s["logits"], out, rows_per_group=s["per"], prompt_tokens=s["prompt_tokens"],
                            cu_prompt=s["cu_prompt"], own_tokens=s["own_tokens"], own_lens=s["own_lens"],
                            repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                            bias_tokens=s["bias_tokens"], bias_values=s["bias_values"], cu_bias=s["cu_bias"],
                            mask=s["mask"], mask_index=s["mask_index"])
        return out
    if op == TREE:
        if "workspace" not in s:                             # kept by the caller, as for the other attention calls
            size = bg.bg_tree_attn_workspace_size(s["cu_nodes"].numel() - 1, s["k"].shape[0], s["max_nodes"],
                                                  s["max_prefix_len"], s["q"].shape[1], s["k"].shape[1], s["q"].shape[2])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["q"].device)
        out = torch.empty_like(s["q"])
        bg.bg_tree_attn(s["q"], s["k"], s["v"], s["parent"], s["cu_nodes"], s["max_nodes"], s["prefix_k"],
                        s["prefix_v"], s["cu_prefix"], s["max_prefix_len"], out, scale=s["scale"],
                        softcap=s["softcap"], workspace=s["workspace"])
        return out
    q, k, v = _split(s)
    kw = {"q_weight": s["q_weight"], "k_weight": s["k_weight"], "eps": s["eps"], "inv_freq": s["inv_freq"],
          "axis_of": s["axis_of"], "interleaved": s["interleaved"]}
    out = {"q": torch.empty(q.shape, dtype=q.dtype, device=q.device)}
    if op == ROPE:
        out["k"], out["v"] = (torch.empty(k.shape, dtype=k.dtype, device=k.device) for _ in range(2))
        bg.bg_packed_qk_norm_rope(q, k, v, s["positions"], out["q"], out["k"], out["v"], **kw)
        return out
    rw = (s["requests"], s["width"])
    out["q"] = out["q"].unflatten(0, rw)
    bg.bg_beam_qk_norm_rope(q.unflatten(0, rw), k.unflatten(0, rw), v.unflatten(0, rw), s["base_pos"], s["step"],
                            out["q"], s["suffix_k"], s["suffix_v"], s["slot"], **kw)
    return dict(out, k=s["suffix_k"], v=s["suffix_v"])


# --------------------------------------------------------------------------- work
def work(case):
    """Each input read once and each output written once; logits only where the mask allows them, and the beams'
    suffix only at the slot that is written."""
    op = case["op"]
    if op in (ROPE, BEAM):
        rows = case["tokens"] if op == ROPE else case["requests"] * case["width"]
        heads, d = case["hq"] + case["hkv"], case["d"]
        places = case["axes"] * (rows if op == ROPE else case["requests"])
        # per element of q and k: the square and its sum, the norm's two products, the rotation's multiply-adds
        return {"bytes": 4 * rows * d * (heads + case["hkv"]) + 4 * places + 2 * case["rot"] + 4 * d * case["norm"],
                "flops": rows * heads * (4 * d * case["norm"] + 3 * case["rot"])}
    if op == LOGITS:
        rows, vocab = case["groups"] * case["per"], case["vocab"]
        n, es = rows * vocab, 4 if case["dtype"] == "float32" else 2
        read = case["allowed"] + (1 - case["allowed"]) / 32 if case["masks"] else 1.0
        mask = case["masks"] * ((vocab + 31) // 32) * 4
        lists = 4 * (case["groups"] * (case["prompt"] * 3 // 4 + 2 * case["bias"] + 5) + rows * (case["own_len"] * 3 // 4 + 2))
        return {"bytes": int(n * es * read) + 4 * n + mask + lists, "flops": int(4 * n * read)}
    nodes, prefix = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    # of the drafted nodes a token sees a path; counted as the largest depth a balanced draft would have
    pairs = sum(n * (p + min(n, 8)) for n, p in zip(nodes, prefix))
    rows = sum(nodes)
    return {"bytes": 2 * d * (2 * rows * hq + 2 * hkv * (rows + sum(prefix))) + 4 * rows, "flops": 4 * d * hq * pairs}


# --------------------------------------------------------------------------- definition in 64 bits
def _exact_rope(s):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    half = s["inv_freq"].numel()
    x = s["qkv"].view(-1, hq + 2 * hkv, d)
    rows = x.shape[0]
    if s["op"] == ROPE:
        pos = s["positions"].double()
    else:
        pos = (s["base_pos"].double() + s["step"])[:, :, None].expand(-1, -1, s["width"]).reshape(-1, rows)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for h0 in range(0, hq + 2 * hkv, 8):                     # a few heads at a time
        out[:, h0:h0 + 8] = x[:, h0:h0 + 8].double()
    for w, a, b in ((s["q_weight"], 0, hq), (s["k_weight"], hq, hq + hkv)):
        if w is not None:
            y = out[:, a:b]
            y.mul_(torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"])).mul_(w.double())
    for i in range(half):                                    # a pair of dimensions at a time, as a complex number
        lo, hi = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        axis = 0 if s["axis_of"] is None else s["axis_of"][i]
        turn = torch.polar(torch.ones_like(pos[axis]), pos[axis] * float(s["inv_freq"][i]))[:, None]
        z = torch.complex(out[:, :hq + hkv, lo], out[:, :hq + hkv, hi]) * turn
        out[:, :hq + hkv, lo], out[:, :hq + hkv, hi] = z.real, z.imag
    q, k, v = out.split((hq, hkv, hkv), 1)
    if s["op"] == ROPE:
        return {"q": q, "k": k, "v": v}
    rw = (s["requests"], s["width"])
    sk, sv = s["suffix_k"].double(), s["suffix_v"].double()
    sk[:, :, s["slot"]], sv[:, :, s["slot"]] = k.unflatten(0, rw), v.unflatten(0, rw)
    return {"q": q.unflatten(0, rw), "k": sk, "v": sv}


def _exact_logits(s):
    out = s["logits"].double()
    rows, vocab = out.shape
    cup, lens = s["cu_prompt"].tolist(), s["own_lens"].tolist()
    index = s["mask_index"].tolist() if s["mask"] is not None else None
    shifts = torch.arange(32, device=out.device)
    for i in range(rows):                                    # one row at a time
        g = i // s["per"]
        row = out[i]
        own_count = torch.bincount(s["own_tokens"][i, :lens[i]].long(), minlength=vocab)
        hit = torch.cat((s["prompt_tokens"][cup[g]:cup[g + 1]], s["own_tokens"][i, :lens[i]])).long().unique()
        rho = s["repetition"][g].double()
        row[hit] = torch.where(row[hit] > 0, row[hit] / rho, row[hit] * rho)
        used = own_count.nonzero()[:, 0]
        row[used] -= s["frequency"][g].double() * own_count[used] + s["presence"][g].double()
        if s["bias_tokens"] is not None:
            a, b = s["cu_bias"][g], s["cu_bias"][g + 1]
            row[s["bias_tokens"][a:b].long()] += s["bias_values"][a:b].double()
        if index is not None and index[i] >= 0:
            bits = (s["mask"][index[i]].long()[:, None] >> shifts) & 1
            row[bits.flatten()[:vocab] == 0] = -math.inf
    return out


def _exact_tree(s):
    cun, cup, parent = s["cu_nodes"].tolist(), s["cu_prefix"].tolist(), s["parent"].tolist()
    hq, hkv = s["q"].shape[1], s["k"].shape[1]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for r in range(len(cun) - 1):
        a, n, p0, p1 = cun[r], cun[r + 1] - cun[r], cup[r], cup[r + 1]
        hidden = torch.ones((n, n), dtype=torch.bool)
        for i in range(n):
            j = i
            while j >= 0:                                    # the node and its ancestors
                hidden[i, j] = False
                j = parent[a + j]
        hidden = hidden.cuda()
        for h in range(hkv):
            k = torch.cat((s["prefix_k"][p0:p1, h], s["k"][a:a + n, h])).double()
            v = torch.cat((s["prefix_v"][p0:p1, h], s["v"][a:a + n, h])).double()
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            x = torch.einsum("nhd,kd->hnk", s["q"][a:a + n, heads].double(), k) * s["scale"]
            if s["softcap"]:
                x = s["softcap"] * torch.tanh(x / s["softcap"])
            x[:, :, p1 - p0:].masked_fill_(hidden, -math.inf)
            out[a:a + n, heads] = torch.einsum("hnk,kd->nhd", torch.softmax(x, -1), v)
    return out


def exact(case, seed):
    op = case["op"]
    if op == ROPE and case["tokens"] * (case["hq"] + 2 * case["hkv"]) * case["d"] > 1 << 29:
        return None
    s = prepare(case, seed)
    return {ROPE: _exact_rope, BEAM: _exact_rope, LOGITS: _exact_logits, TREE: _exact_tree}[op](s)
