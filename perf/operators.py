"""Cases that measure the attention-side operators of a decoder layer: rotary
positions, the quantised paged key/value cache (written and read back),
attention over prompts and attention of single tokens over the cache.

``run`` computes an operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end), or, where ``own`` is true, with the
calls a user makes of this framework.  ``exact`` gives the same outputs from
the definitions in 64 bits.

Head counts and sizes are those of the framework's workloads: the 27B-class
decoder (40 query heads, 8 key/value heads, head dimension 128) and the 0.6B
embedding model (16 query heads, 8 key/value heads, head dimension 128).
"""
import math
import random

import torch

own = False

X_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3_MAX, I8_MAX = 448.0, 127.0


# --------------------------------------------------------------------- cases

def listed():
    return [
        # One decoding step of 16 sequences of the 27B-class decoder: positions
        # of one new token each, where the launch is what counts.
        {"name": "rope_step_16", "op": "rope", "tokens": 16, "q_heads": 40, "kv_heads": 8, "dim": 128,
         "rot": 128, "layout": "half", "factor": 1.0, "type": "bf16"},
        # A long prompt: half of each head rotated, interleaved pairs,
        # frequencies scaled to four times the trained context.
        {"name": "rope_prompt_8191", "op": "rope", "tokens": 8191, "q_heads": 40, "kv_heads": 8, "dim": 128,
         "rot": 64, "layout": "interleaved", "factor": 4.0, "type": "f16"},
        # The cache side of one decoding step of 16 sequences: rotate, quantise
        # and store one token each, and read those tokens back.
        {"name": "cache_step_16_e4m3", "op": "cache", "tokens": 16, "q_heads": 40, "kv_heads": 8, "dim": 128,
         "rot": 128, "layout": "half", "factor": 1.0, "type": "bf16", "kv": "e4m3", "page": 16},
        # The cache side of a long prompt of odd length, and the read of all of
        # it that precedes the attention of the prompt's next part.
        {"name": "cache_prompt_8191_i8", "op": "cache", "tokens": 8191, "q_heads": 40, "kv_heads": 8, "dim": 128,
         "rot": 128, "layout": "half", "factor": 4.0, "type": "bf16", "kv": "i8", "page": 64},
        # A packed batch of short search queries through the embedding model.
        {"name": "prompt_queries_32", "op": "prompt", "seqs": 32, "longest": 48, "past": 0, "lens": 1, "spread": True,
         "q_heads": 16, "kv_heads": 8, "dim": 128, "causal": True, "type": "bf16"},
        # A packed batch of documents of unequal length through the embedding
        # model, each token attending to its whole document.
        {"name": "prompt_documents_24", "op": "prompt", "seqs": 24, "longest": 1023, "past": 0, "lens": 2, "spread": True,
         "q_heads": 16, "kv_heads": 8, "dim": 128, "causal": False, "type": "f16"},
        # One long prompt of the 27B-class decoder.
        {"name": "prompt_8192", "op": "prompt", "seqs": 1, "longest": 8192, "past": 0, "lens": 3, "spread": False,
         "q_heads": 40, "kv_heads": 8, "dim": 128, "causal": True, "type": "bf16"},
        # The last part of a long prompt that is worked through in parts: few
        # new tokens against many that are in the cache already.
        {"name": "prompt_part_256_of_16384", "op": "prompt", "seqs": 1, "longest": 256, "past": 16128, "lens": 4,
         "spread": False, "q_heads": 40, "kv_heads": 8, "dim": 128, "causal": True, "type": "bf16"},
        # One short conversation, cache of 16-bit values.
        {"name": "token_1_of_701", "op": "token", "seqs": 1, "longest": 701, "lens": 5, "spread": False,
         "q_heads": 40, "kv_heads": 8, "dim": 128, "type": "bf16", "kv": "x16", "page": 16},
        # A serving batch of unequal conversations (one of them idle, of length
        # zero), 8-bit floating-point cache.
        {"name": "token_32_to_8192_e4m3", "op": "token", "seqs": 32, "longest": 8192, "lens": 6, "spread": True,
         "q_heads": 40, "kv_heads": 8, "dim": 128, "type": "bf16", "kv": "e4m3", "page": 16},
        # Few very long conversations, 16-bit cache: the length has to be split.
        {"name": "token_2_of_32768", "op": "token", "seqs": 2, "longest": 32768, "lens": 7, "spread": False,
         "q_heads": 40, "kv_heads": 8, "dim": 128, "type": "f16", "kv": "x16", "page": 64},
        # A full serving batch, 8-bit integer cache.
        {"name": "token_128_of_8192_i8", "op": "token", "seqs": 128, "longest": 8192, "lens": 8, "spread": False,
         "q_heads": 40, "kv_heads": 8, "dim": 128, "type": "bf16", "kv": "i8", "page": 32},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "prompt", "prompt", "token", "token"])
    q_heads, kv_heads = rng.choice([(40, 8), (16, 8), (32, 4), (8, 8), (24, 2), (12, 1)])
    case = {"op": op, "q_heads": q_heads, "kv_heads": kv_heads, "dim": rng.choice([128, 128, 128, 64, 96, 80]),
            "type": rng.choice(["bf16", "bf16", "f16"])}
    if op in ("rope", "cache"):
        case["tokens"] = _log(rng, 1, 8191)
        case["rot"] = rng.choice([case["dim"], case["dim"], case["dim"] // 2])
        case["layout"] = rng.choice(["half", "interleaved"])
        case["factor"] = rng.choice([1.0, 4.0, 8.0])
        if op == "cache":
            case["kv"] = rng.choice(["e4m3", "i8", "x16"])
            case["page"] = rng.choice([16, 32, 64, 128])
    elif op == "prompt":
        case["seqs"] = _log(rng, 1, 24)
        case["causal"] = rng.random() < 0.7
        # the longest listed prompt has 8192 x 8192 scores of 40 heads, half of them seen
        most = math.sqrt(8192.0 * 8192.0 * 40 * (1.0 if case["causal"] else 0.5) / (q_heads * case["seqs"]))
        case["longest"] = _log(rng, 1, max(2, min(8192, int(most))))
        case["past"] = rng.choice([0, 0, _log(rng, 1, 2048)])
        case["past"] = min(case["past"], max(0, int(most * most / case["longest"]) - case["longest"]))
        case["lens"] = rng.randrange(1 << 20)
        case["spread"] = case["seqs"] > 1
    else:
        case["kv"] = rng.choice(["e4m3", "i8", "x16"])
        case["page"] = rng.choice([16, 32, 64, 128])
        case["seqs"] = _log(rng, 1, 128)
        # the largest listed batch holds 128 x 8192 tokens of 8 heads in 8 bits
        most = 128 * 8192 * 8 * 128 // (case["seqs"] * kv_heads * case["dim"] * (2 if case["kv"] == "x16" else 1))
        case["longest"] = _log(rng, 1, max(2, min(32768, most)))
        case["lens"] = rng.randrange(1 << 20)
        case["spread"] = rng.random() < 0.7 and case["seqs"] > 1
    return case


def _lengths(case):
    """New tokens of each sequence, and tokens it has in all.  Unequal lengths
    are spread over their logarithm; one sequence in sixteen is idle."""
    rng = random.Random(case["lens"])
    n, longest = case["seqs"], case["longest"]
    if case["spread"]:
        new = [_log(rng, max(1, longest // 32), longest) for _ in range(n)]
        new[rng.randrange(n)] = longest
        for i in range(n // 16):
            new[(5 + 16 * i) % n] = 0
    else:
        new = [longest] * n
    past = case.get("past", 0)
    if past and case["spread"]:
        return new, [x + rng.randrange(past + 1) for x in new]
    return new, [x + past for x in new]


def work(case):
    """Inputs read once, outputs written once; products of the pairs that attend."""
    h, g, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        t = case["tokens"]
        return {"bytes": t * (h + g) * d * 4 + 4 * t + 2 * case["rot"], "flops": 3 * t * (h + g) * case["rot"]}
    if case["op"] == "cache":
        t = case["tokens"]
        cell = 2 * d if case["kv"] == "x16" else d + 4
        # q in and out; k and v in, stored, and out again
        return {"bytes": t * (h * d * 4 + 2 * g * (4 * d + cell)) + 20 * t, "flops": t * ((h + g) * 3 * case["rot"] + 6 * g * d)}
    new, total = _lengths(case)
    if case["op"] == "prompt":
        pairs = 0
        for q, k in zip(new, total):
            # row i of q attends to the first k - q + i + 1 keys, or to all k
            pairs += q * k - (q * (q - 1)) // 2 if case["causal"] else q * k
        return {"bytes": sum(new) * h * (4 * d + 4) + sum(total) * g * d * 4, "flops": 4 * pairs * h * d}
    cell = 2 * d if case["kv"] == "x16" else d + 4
    return {"bytes": sum(total) * g * 2 * cell + case["seqs"] * h * (4 * d + 4), "flops": 4 * sum(total) * h * d}


# -------------------------------------------------------------------- inputs

def _device():
    return torch.device("cuda:0") if torch.cuda.is_available() else torch.device("cpu")


def _frequencies(rot, factor, dev):
    """Rotation per position of each pair, base 1e6.  With a factor above 1,
    pairs that turn less than once over the trained context are slowed down by
    it, those that turn 32 times or more are kept, with a ramp between; the
    rotated values grow by 0.1 ln(factor) + 1."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 1e6 ** (-2.0 * i / rot)
    if factor <= 1.0:
        return f.float().to(dev), 1.0
    turns = 32768.0 / factor * f / (2 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return (f * keep + f / factor * (1 - keep)).float().to(dev), 0.1 * math.log(factor) + 1.0


def _heads(g, dev, rows, heads, dim, dtype, spread):
    """Projections as a layer makes them: every channel of a head has a size of
    its own (a few are several times the others), values are normal."""
    size = torch.exp(spread * torch.randn((1, heads, dim), generator=g, device=dev))
    return (torch.randn((rows, heads, dim), generator=g, device=dev) * size).to(dtype)


def _quantised(x, kv):
    """8-bit codes and the fp32 factor of each run of `dim` values."""
    top = I8_MAX if kv == "i8" else E4M3_MAX
    x = x.float()
    most = x.abs().amax(-1, keepdim=True)
    inv = torch.where(most > 0, top / most, torch.zeros_like(most))
    y = x * inv
    code = torch.round(y).to(torch.int8) if kv == "i8" else y.clamp(-top, top).to(torch.float8_e4m3fn)
    return code, (most / top).squeeze(-1)


def _cache_type(case):
    return {"x16": X_TYPES[case["type"]], "i8": torch.int8, "e4m3": torch.float8_e4m3fn}[case["kv"]]


def _workspace(kind, *sizes):
    from ternary_bit_weight_gb300 import binding as tb
    n = getattr(tb, kind)(*sizes)
    return torch.zeros(n, dtype=torch.uint8, device=_device())


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * int(seed) + 17)
    x = X_TYPES[case["type"]]
    h, g, d = case["q_heads"], case["kv_heads"], case["dim"]
    s = {"case": case}
    if case["op"] in ("rope", "cache"):
        t = case["tokens"]
        s["inv_freq"], s["amplitude"] = _frequencies(case["rot"], case["factor"], dev)
        if t <= 256:   # a decoding step: a position of its own for every sequence
            s["pos"] = torch.randint(0, 32768, (t,), generator=gen, device=dev, dtype=torch.int32)
        else:          # a prompt
            s["pos"] = torch.arange(t, device=dev, dtype=torch.int32) + 24000
        # the fused projection's output: q, k and v of a token beside one another
        s["qkv"] = torch.cat([_heads(gen, dev, t, h, d, x, 0.4), _heads(gen, dev, t, g, d, x, 0.4),
                              _heads(gen, dev, t, g, d, x, 0.2)], 1)
        s["q"] = torch.empty((t, h, d), dtype=x, device=dev)
        s["k"] = torch.empty((t, g, d), dtype=x, device=dev)
        if case["op"] == "cache":
            s["v"] = torch.empty((t, g, d), dtype=x, device=dev)
            pages = -(-t // case["page"]) + 3 if t > 256 else t + 3
            order = torch.randperm(pages, generator=gen, device=dev)
            at = torch.arange(t, device=dev)
            if t > 256:
                s["slots"] = order[at // case["page"]] * case["page"] + at % case["page"]
            else:      # every sequence in a page of its own
                s["slots"] = order[:t] * case["page"] + torch.randint(0, case["page"], (t,), generator=gen, device=dev)
            s["pages"] = pages
            shape = (pages, g, case["page"], d)
            s["k_cache"] = torch.zeros(shape, dtype=torch.uint8, device=dev).to(_cache_type(case))
            s["v_cache"] = torch.zeros(shape, dtype=torch.uint8, device=dev).to(_cache_type(case))
            s["k_scale"] = torch.zeros(shape[:3], dtype=torch.float32, device=dev)
            s["v_scale"] = torch.zeros(shape[:3], dtype=torch.float32, device=dev)
        return s
    new, total = _lengths(case)
    if case["op"] == "prompt":
        nq, nk = sum(new), sum(total)
        s["q_max"], s["k_max"] = max(new), max(total)
        cum = torch.tensor([[sum(new[:i]), sum(total[:i])] for i in range(len(new) + 1)], dtype=torch.int32, device=dev)
        s["cu_q"], s["cu_k"] = cum[:, 0].contiguous(), cum[:, 1].contiguous()
        s["q"] = _heads(gen, dev, nq, h, d, x, 0.4)
        s["k"] = _heads(gen, dev, nk, g, d, x, 0.4)
        s["v"] = _heads(gen, dev, nk, g, d, x, 0.2)
        s["o"] = torch.empty((nq, h, d), dtype=x, device=dev)
        s["lse"] = torch.empty((nq, h), dtype=torch.float32, device=dev)
        if own:
            s["ws"] = _workspace("tern_attn_prompt_workspace_bytes", len(new), nq, nk, h, g, d)
        return s
    page, n = case["page"], case["seqs"]
    per = -(-max(total) // page)
    pages = n * per + 5
    shape = (pages, g, page, d)
    s["per"], s["pages"] = per, pages
    s["table"] = torch.randperm(pages, generator=gen, device=dev)[:n * per].to(torch.int32).reshape(n, per)
    s["lens"] = torch.tensor(total, dtype=torch.int32, device=dev)
    s["q"] = _heads(gen, dev, n, h, d, x, 0.4)
    for name, spread in (("k", 0.4), ("v", 0.2)):
        c = _heads(gen, dev, pages * page, g, d, x, spread).reshape(pages, page, g, d).transpose(1, 2)
        if case["kv"] == "x16":
            s[name + "_cache"], s[name + "_scale"] = c.contiguous(), None
        else:
            s[name + "_cache"], s[name + "_scale"] = (y.contiguous() for y in _quantised(c, case["kv"]))
        del c
    s["o"] = torch.empty((n, h, d), dtype=x, device=dev)
    s["lse"] = torch.empty((n, h), dtype=torch.float32, device=dev)
    if own:
        s["ws"] = _workspace("tern_attn_decode_workspace_bytes", n, h, g, d, per * page)
    return s


# --------------------------------------------------------------- plain forms

def _rotated(x, s, angle):
    """Heads [t, h, d] rotated by angle [t, rot/2], in x's own precision."""
    case = s["case"]
    rot = case["rot"]
    c, n = (angle.cos() * s["amplitude"])[:, None], (angle.sin() * s["amplitude"])[:, None]
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(s):
    h, g = s["case"]["q_heads"], s["case"]["kv_heads"]
    x = s["qkv"].dtype
    angle = s["pos"].float()[:, None] * s["inv_freq"]
    qk = _rotated(s["qkv"][:, :h + g].float(), s, angle)
    return qk[:, :h].to(x), qk[:, h:].to(x)


def _plain_cache(s):
    case = s["case"]
    h, g, page, x = case["q_heads"], case["kv_heads"], case["page"], s["qkv"].dtype
    q, k = _plain_rope(s)
    at, row = s["slots"] // page, s["slots"] % page
    out = [q]
    for name, new in (("k", k), ("v", s["qkv"][:, h + g:])):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        if case["kv"] == "x16":
            cache[at, :, row] = new
            out.append(cache[at, :, row])
        else:
            code, factor = _quantised(new, case["kv"])
            cache.view(torch.uint8)[at, :, row] = code.view(torch.uint8)
            scale[at, :, row] = factor
            code = cache.view(torch.uint8)[at, :, row].view(cache.dtype)
            out.append((code.float() * scale[at, :, row][..., None]).to(x))
    return {"q": out[0], "k": out[1], "v": out[2]}


def _plain_attention(q, k, v, seen, scale):
    """q [b, g, r, d], k and v [b, g, l, d] in 32 bits, seen [b, 1, r or 1, l]
    -> outputs [b, g, r, d] and the logarithms of the sums [b, g, r]; a row
    that sees nothing is zero, with logarithm minus infinity."""
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    p = p.masked_fill_(~seen, float("-inf"))
    most = p.amax(-1, keepdim=True)
    most = torch.where(torch.isinf(most), torch.zeros_like(most), most)
    p = p.sub_(most).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o, (most + total.log()).squeeze(-1)


def _padded(x, cu, most):
    """Packed rows [t, ...] as [sequences, most, ...], and which of them exist."""
    at = torch.arange(most, device=x.device)
    there = at < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None].long() + at).clamp_(max=max(0, x.shape[0] - 1))
    return x[rows], there


def _plain_prompt(s):
    case = s["case"]
    h, g, d = case["q_heads"], case["kv_heads"], case["dim"]
    q, q_there = _padded(s["q"], s["cu_q"], s["q_max"])
    k, k_there = _padded(s["k"], s["cu_k"], s["k_max"])
    v, _ = _padded(s["v"], s["cu_k"], s["k_max"])
    b, r, l = q.shape[0], s["q_max"], s["k_max"]
    seen = k_there[:, None, None, :]
    if case["causal"]:
        shift = (s["cu_k"][1:] - s["cu_k"][:-1]) - (s["cu_q"][1:] - s["cu_q"][:-1])
        i, j = torch.arange(r, device=q.device), torch.arange(l, device=q.device)
        seen = seen & (j <= i[:, None] + shift[:, None, None])[:, None]
        seen = seen.repeat(1, 1, h // g, 1)
    # the query heads that share a key/value head are rows of one product
    q = q.float().reshape(b, r, g, h // g, d).permute(0, 2, 3, 1, 4).reshape(b, g, h // g * r, d)
    k, v = k.float().transpose(1, 2), v.float().transpose(1, 2)
    o, lse = _plain_attention(q, k, v, seen, 1.0 / math.sqrt(d))
    o = o.reshape(b, g, h // g, r, d).permute(0, 3, 1, 2, 4).reshape(b, r, h, d)
    lse = lse.reshape(b, g, h // g, r).permute(0, 3, 1, 2).reshape(b, r, h)
    return {"o": o[q_there].to(s["q"].dtype), "lse": lse[q_there]}


def _plain_token(s):
    case = s["case"]
    h, g, d, n = case["q_heads"], case["kv_heads"], case["dim"], case["seqs"]
    l = s["per"] * case["page"]
    table = s["table"].long()
    kv = []
    for name in ("k", "v"):
        c = s[name + "_cache"]
        c = c[table] if c.dtype != torch.float8_e4m3fn else c.view(torch.uint8)[table].view(c.dtype)
        c = c.float()
        if s[name + "_scale"] is not None:
            c = c * s[name + "_scale"][table][..., None]
        kv.append(c.transpose(1, 2).reshape(n, g, l, d))
    seen = (torch.arange(l, device=table.device) < s["lens"][:, None])[:, None, None]
    o, lse = _plain_attention(s["q"].float().reshape(n, g, h // g, d), *kv, seen, 1.0 / math.sqrt(d))
    return {"o": o.reshape(n, h, d).to(s["q"].dtype), "lse": lse.reshape(n, h)}


# ------------------------------------------------------ the framework's calls

def _own(s):
    from ternary_bit_weight_gb300 import binding as tb
    case = s["case"]
    op, h, g, d = case["op"], case["q_heads"], case["kv_heads"], case["dim"]
    x = tb.TERN_X_BF16 if case["type"] == "bf16" else tb.TERN_X_F16
    if op in ("rope", "cache"):
        layout = tb.TERN_ROPE_HALF if case["layout"] == "half" else tb.TERN_ROPE_INTERLEAVED
        t, qkv = case["tokens"], s["qkv"]
        ld = (h + 2 * g) * d
        q, k, v = qkv, qkv.data_ptr() + 2 * h * d, qkv.data_ptr() + 2 * (h + g) * d
    if op == "rope":
        tb.tern_rope(x, layout, t, d, case["rot"], s["pos"], s["inv_freq"], s["amplitude"],
                     h, q, ld, s["q"], h * d, g, k, ld, s["k"], g * d)
        return s["q"], s["k"]
    if op in ("cache", "token"):
        kv = {"x16": tb.TERN_KV_X16, "e4m3": tb.TERN_KV_E4M3, "i8": tb.TERN_KV_I8}[case["kv"]]
        cache = (s["pages"], case["page"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if op == "cache":
        tb.tern_rope_kv_write(x, kv, layout, t, h, g, d, case["rot"], s["pos"], s["inv_freq"], s["amplitude"],
                              q, ld, s["q"], h * d, k, ld, v, ld, s["slots"], *cache)
        tb.tern_kv_read(x, kv, t, g, d, s["slots"], *cache, s["k"], g * d, s["v"], g * d)
        return {"q": s["q"], "k": s["k"], "v": s["v"]}
    if op == "prompt":
        tb.tern_attn_prompt(x, case["seqs"], s["cu_q"], s["cu_k"], s["q"].shape[0], s["k"].shape[0], h, g, d,
                            case["causal"], 1.0 / math.sqrt(d), s["q"], h * d, s["k"], g * d, s["v"], g * d,
                            s["o"], h * d, s["lse"], s["ws"])
    else:
        tb.tern_attn_decode(x, kv, case["seqs"], h, g, d, 1.0 / math.sqrt(d), s["q"], h * d, *cache,
                            s["table"], s["per"], s["lens"], s["o"], h * d, s["lse"], s["ws"])
    return {"o": s["o"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"rope": _plain_rope, "cache": _plain_cache, "prompt": _plain_prompt, "token": _plain_token}[op](state)


# ------------------------------------------------------------------- 64 bits

def _exact_rope(s):
    """Each pair as a complex number times amplitude * exp(i * angle)."""
    case = s["case"]
    h, g, rot = case["q_heads"], case["kv_heads"], case["rot"]
    turn = torch.polar(torch.full_like(s["inv_freq"].double(), s["amplitude"]).expand(case["tokens"], -1).contiguous(),
                       torch.outer(s["pos"].double(), s["inv_freq"].double()))
    y = s["qkv"][:, :h + g].double()
    part = y[..., :rot]
    if case["layout"] == "half":
        z = torch.complex(*part.split(rot // 2, -1)) * turn[:, None]
        y[..., :rot] = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(part.reshape(*part.shape[:-1], rot // 2, 2).contiguous()) * turn[:, None]
        y[..., :rot] = torch.view_as_real(z).reshape(part.shape)
    return y[:, :h], y[:, h:]


def _exact_rows(q, k, v, scale):
    """One group of query rows that see all of k: softmax by its definition."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full(q.shape[:1], float("-inf"), dtype=torch.float64, device=q.device)
    z = q @ k.T * scale
    lse = torch.logsumexp(z, -1)
    return torch.exp(z - lse[:, None]) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    h, g, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "cache":
        # what the codes stand for is an approximation of these values
        q, k = _exact_rope(s)
        return {"q": q, "k": k, "v": s["qkv"][:, h + g:].double()}
    if work(case)["flops"] > 3e12:
        return None
    scale = 1.0 / math.sqrt(d)
    new, total = _lengths(case)
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=s["o"].device)
    lse = torch.full(s["lse"].shape, float("-inf"), dtype=torch.float64, device=o.device)
    if case["op"] == "prompt":
        q_at = k_at = 0
        for nq, nk in zip(new, total):
            for head in range(h):
                q = s["q"][q_at:q_at + nq, head].double()
                k = s["k"][k_at:k_at + nk, head // (h // g)].double()
                v = s["v"][k_at:k_at + nk, head // (h // g)].double()
                z = q @ k.T * scale
                if case["causal"]:
                    z = z.masked_fill(torch.ones_like(z, dtype=torch.bool).triu(1 + nk - nq), float("-inf"))
                e = torch.logsumexp(z, -1) if nk else torch.full((nq,), float("-inf"), dtype=torch.float64, device=z.device)
                p = torch.exp(z - torch.where(torch.isinf(e), torch.zeros_like(e), e)[:, None])
                o[q_at:q_at + nq, head] = p @ v
                lse[q_at:q_at + nq, head] = e
            q_at, k_at = q_at + nq, k_at + nk
        return {"o": o, "lse": lse}
    for b, n in enumerate(total):
        pages = s["table"][b, :-(-n // case["page"])].long() if n else s["table"][b, :0].long()
        kv = []
        for name in ("k", "v"):
            c = s[name + "_cache"].view(torch.uint8)[pages].view(s[name + "_cache"].dtype).double()
            if s[name + "_scale"] is not None:
                c = c * s[name + "_scale"][pages].double()[..., None]
            kv.append(c.transpose(0, 1).reshape(g, -1, d)[:, :n])
        for head in range(g):
            rows = slice(head * (h // g), (head + 1) * (h // g))
            o[b, rows], lse[b, rows] = _exact_rows(s["q"][b, rows].double(), kv[0][head], kv[1][head], scale)
    return {"o": o, "lse": lse}
