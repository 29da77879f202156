"""Cases that measure the norm at a decoder layer's two ends (with the residual's
addition, and with 8-bit outputs for the int8 linear), and what keeps a paged
key/value cache within a budget: the attention weight each cached token has
received, the choice of the tokens to keep, and their move to the front.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end), or, where ``own`` is true, with the calls a
user makes of this framework.  ``exact`` gives the same outputs from the
definitions in 64 bits.

Head counts and sizes are those of the framework's workloads: the 27B-class
decoder (hidden size 5120, 27648 inside the MLP, 40 query heads, 8 key/value
heads, head dimension 128) and the 0.6B embedding model (hidden size 1024, 16
query heads, 8 key/value heads, head dimension 128).
"""
import math
import random

import numpy as np
import torch

own = False

X_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# --------------------------------------------------------------------- cases

def listed():
    return [
        # One decoding step of 16 sequences of the 27B-class decoder: the attention's
        # output joins the residual stream and is normalised for the MLP.
        {"name": "norm_step_16", "op": "norm", "tokens": 16, "heads": 1, "size": 5120, "type": "bf16", "in": "bf16",
         "res": "bf16", "add": 0.0, "out": "x16"},
        # The same for a long prompt of odd length, the linear's fp32 output added to
        # the stream and the result quantised for the int8 linear.
        {"name": "norm_prompt_8191_i8", "op": "norm", "tokens": 8191, "heads": 1, "size": 5120, "type": "bf16",
         "in": "f32", "res": "bf16", "add": 0.0, "out": "i8"},
        # The query heads of a prompt, each normalised by itself, in the fused
        # projection's output.
        {"name": "norm_heads_4095", "op": "norm", "tokens": 4095, "heads": 40, "size": 128, "type": "bf16", "in": "bf16",
         "res": "none", "add": 1.0, "out": "x16"},
        # One short conversation: the weights of its newest token.
        {"name": "weights_token_1_of_701", "op": "weights", "seqs": 1, "longest": 701, "rows": 1, "lens": 1, "spread": False,
         "q_heads": 40, "kv_heads": 8, "dim": 128, "type": "bf16", "kv": "x16", "page": 16, "decay": 1.0},
        # A serving batch of unequal conversations (some of them idle, of length
        # zero), 8-bit floating-point cache, weights that fade.
        {"name": "weights_token_32_to_8192_e4m3", "op": "weights", "seqs": 32, "longest": 8192, "rows": 1, "lens": 2,
         "spread": True, "q_heads": 40, "kv_heads": 8, "dim": 128, "type": "bf16", "kv": "e4m3", "page": 16, "decay": 0.98},
        # A full serving batch, 8-bit integer cache.
        {"name": "weights_token_128_of_8192_i8", "op": "weights", "seqs": 128, "longest": 8192, "rows": 1, "lens": 3,
         "spread": False, "q_heads": 40, "kv_heads": 8, "dim": 128, "type": "bf16", "kv": "i8", "page": 32, "decay": 1.0},
        # Prompts just worked through, judged by what their last 32 tokens attend to.
        {"name": "weights_window_4x32_of_8191", "op": "weights", "seqs": 4, "longest": 8191, "rows": 32, "lens": 4,
         "spread": False, "q_heads": 40, "kv_heads": 8, "dim": 128, "type": "bf16", "kv": "x16", "page": 64, "decay": 1.0},
        # A prompt judged by all of its tokens.
        {"name": "weights_prompt_4096", "op": "weights", "seqs": 1, "longest": 4096, "rows": 4096, "lens": 5,
         "spread": False, "q_heads": 40, "kv_heads": 8, "dim": 128, "type": "bf16", "kv": "x16", "page": 16, "decay": 1.0},
        # One conversation that has outgrown its budget by an eighth.
        {"name": "keep_512_of_577", "op": "keep", "seqs": 1, "longest": 577, "lens": 6, "spread": False, "kv_heads": 8,
         "page": 16, "budget": 512, "first": 4, "recent": 64},
        # A serving batch brought down to half its length.
        {"name": "keep_4096_of_8192", "op": "keep", "seqs": 64, "longest": 8192, "lens": 7, "spread": False, "kv_heads": 8,
         "page": 32, "budget": 4096, "first": 4, "recent": 256},
        # The moves of one such conversation, 8-bit cache.
        {"name": "compact_512_of_577_e4m3", "op": "compact", "seqs": 1, "longest": 577, "lens": 8, "spread": False,
         "kv_heads": 8, "dim": 128, "type": "bf16", "kv": "e4m3", "page": 16, "budget": 512, "first": 4, "recent": 64,
         "to": "same"},
        # The moves of such a batch, 16-bit cache.
        {"name": "compact_4096_of_8192", "op": "compact", "seqs": 32, "longest": 8192, "lens": 9, "spread": False,
         "kv_heads": 8, "dim": 128, "type": "bf16", "kv": "x16", "page": 32, "budget": 4096, "first": 4, "recent": 256,
         "to": "same"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "weights", "weights", "weights", "keep", "compact"])
    if op == "norm":
        case = {"op": op, "tokens": _log(rng, 1, 8191), "heads": 1, "type": rng.choice(["bf16", "bf16", "f16"]),
                "add": rng.choice([0.0, 0.0, 1.0])}
        case["out"] = rng.choice(["x16", "x16", "i8"])
        if rng.random() < 0.25:
            case |= {"heads": rng.choice([40, 16, 8, 5]), "size": rng.choice([128, 64, 96, 80, 256]), "in": case["type"],
                     "res": "none", "out": "x16"}
        else:
            # the int8 linear takes whole groups of 128
            case["size"] = (128 * _log(rng, 1, 216) if case["out"] == "i8"
                            else rng.choice([5120, 1024, 27648, 8 * _log(rng, 1, 3456)]))
            case["in"] = rng.choice([case["type"], "f32"])
            case["res"] = rng.choice([case["type"], case["type"], "f32", "none"])
        # the listed prompt has 8191 x 5120 values
        case["tokens"] = min(case["tokens"], max(1, 8191 * 5120 // (case["heads"] * case["size"])))
        return case
    q_heads, kv_heads = rng.choice([(40, 8), (16, 8), (32, 4), (8, 8), (24, 2), (12, 1)])
    case = {"op": op, "kv_heads": kv_heads, "page": rng.choice([16, 32, 64, 128]), "lens": rng.randrange(1 << 20)}
    case["seqs"] = _log(rng, 1, 128)
    if op == "keep":
        # the listed batch has 64 x 8192 tokens of 8 heads
        case["longest"] = _log(rng, 1, max(2, min(32768, 64 * 8192 * 8 // (case["seqs"] * kv_heads))))
    else:
        case |= {"dim": rng.choice([128, 128, 128, 64, 96, 80]), "type": rng.choice(["bf16", "bf16", "f16"]),
                 "kv": rng.choice(["e4m3", "i8", "x16"])}
        wide = kv_heads * case["dim"] * (2 if case["kv"] == "x16" else 1)
        if op == "compact":
            case["longest"] = _log(rng, 1, max(2, min(32768, 32 * 8192 * 8 * 256 // (case["seqs"] * wide))))
        else:
            case["q_heads"] = q_heads
            case["decay"] = rng.choice([1.0, 1.0, 0.98])
            case["rows"] = rng.choice([1, 1, 1, _log(rng, 2, 64), _log(rng, 32, 4096)])
            # the listed batch holds 128 x 8192 tokens of 8 heads in 8 bits, the listed
            # prompt 4096 x 4096 scores of 40 heads, half of them seen
            most = min(32768, 128 * 8192 * 8 * 128 // (case["seqs"] * wide))
            if case["rows"] > 1:
                pairs = 4096 * 4096 * 40 // (2 * q_heads * case["seqs"])
                case["rows"] = max(1, min(case["rows"], int(math.sqrt(pairs))))
                most = min(most, max(1, pairs // case["rows"]))
            case["longest"] = _log(rng, 1, max(2, most))
            case["rows"] = min(case["rows"], case["longest"])
    case["spread"] = rng.random() < 0.6 and case["seqs"] > 1
    if op != "weights":
        case["budget"] = max(1, int(case["longest"] * rng.uniform(0.3, 1.05)))
        case["first"] = min(rng.choice([0, 4, 4, 64]), case["budget"] // 2)
        case["recent"] = min(rng.choice([0, 64, 256]), case["budget"] - case["first"])
        if op == "compact":
            case["to"] = rng.choice(["same", "same", "fresh"])
    return case


def _lengths(case):
    """Tokens of each sequence.  Unequal lengths are spread over their
    logarithm; one sequence in sixteen is idle."""
    rng = random.Random(case["lens"])
    n, longest = case["seqs"], case["longest"]
    if not case["spread"]:
        return [longest] * n
    lens = [_log(rng, max(1, longest // 32), longest) for _ in range(n)]
    lens[rng.randrange(n)] = longest
    for i in range(n // 16):
        lens[(5 + 16 * i) % n] = 0
    return lens


def _rows(case):
    """Query rows of each sequence: the newest of its tokens."""
    return [min(case["rows"], n) for n in _lengths(case)]


def _bytes(name):
    return 4 if name == "f32" else 0 if name == "none" else 2


def work(case):
    """Inputs read once, outputs written once; products of the pairs that attend."""
    if case["op"] == "norm":
        n = case["tokens"] * case["heads"] * case["size"]
        res = _bytes(case["res"])
        return {"bytes": n * (_bytes(case["in"]) + 2 * res + (1 if case["out"] == "i8" else 2)) + 2 * case["size"], "flops": 5 * n}
    g, lens = case["kv_heads"], _lengths(case)
    if case["op"] == "keep":
        kept = sum(min(n, case["budget"]) for n in lens)
        # 4 bytes of weight in, 4 of index out, lists whole
        return {"bytes": 4 * g * (sum(n for n in lens if n > case["budget"]) + case["seqs"] * case["budget"]) + 12 * len(lens),
                "flops": g * (sum(lens) + kept)}
    d = case["dim"]
    cell = 2 * d if case["kv"] == "x16" else d + 4
    if case["op"] == "compact":
        # every list read; tokens behind the first ones read and written: key, value and weight
        moved = sum(max(0, min(n, case["budget"]) - case["first"]) for n in lens if n > case["budget"] or case["to"] == "fresh")
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": g * (2 * moved * (2 * cell + 4) + 4 * kept), "flops": g * moved}
    h = case["q_heads"]
    pairs = sum(q * n - q * (q - 1) // 2 for q, n in zip(_rows(case), lens))
    rows = sum(_rows(case))
    return {"bytes": sum(lens) * g * (cell + 8) + rows * h * (2 * d + 4), "flops": 2 * pairs * h * d}


# -------------------------------------------------------------------- inputs

def _device():
    return torch.device("cuda:0") if torch.cuda.is_available() else torch.device("cpu")


def _heads(g, dev, rows, heads, dim, dtype, spread):
    """Projections as a layer makes them: every channel of a head has a size of
    its own (a few are several times the others), values are normal."""
    size = torch.exp(spread * torch.randn((1, heads, dim), generator=g, device=dev))
    return (torch.randn((rows, heads, dim), generator=g, device=dev) * size).to(dtype)


def _quantised(x, kv):
    """8-bit codes and the fp32 factor of each run of `dim` values."""
    top = 127.0 if kv == "i8" else 448.0
    x = x.float()
    most = x.abs().amax(-1, keepdim=True)
    y = x * torch.where(most > 0, top / most, torch.zeros_like(most))
    code = torch.round(y).to(torch.int8) if kv == "i8" else y.clamp(-top, top).to(torch.float8_e4m3fn)
    return code, (most / top).squeeze(-1)


def _scale(dim):
    return float(np.float32(1.0 / math.sqrt(dim)))


def _raw(c):
    """Indexing moves codes as bytes."""
    return c.view(torch.uint8) if c.element_size() == 1 else c


def _cached(cache, scale, pages):
    """Tokens of `pages` in 32 bits: [..., head, tokens of the pages, dim]."""
    c = _raw(cache)[pages].view(cache.dtype).float()
    if scale is not None:
        c = c * scale[pages][..., None]
    c = c.transpose(-4, -3)
    return c.reshape(*c.shape[:-3], c.shape[-3] * c.shape[-2], c.shape[-1])


def _lse(s):
    """What attention reports for the query rows: the logarithm of each row's sum."""
    case = s["case"]
    h, g, d = case["q_heads"], case["kv_heads"], case["dim"]
    out = torch.zeros((sum(s["new"]), h), dtype=torch.float32, device=s["q"].device)
    at = 0
    for b, (q, n) in enumerate(zip(s["new"], s["total"])):
        if q == 0:
            continue
        k = _cached(s["k_cache"], s["k_scale"], s["table"][b, :-(-n // case["page"])].long())[:, :n].to(s["q"].dtype)
        x = s["q"][at:at + q].reshape(q, g, h // g, d).permute(1, 2, 0, 3)
        # no more than a few GB of scores at a time
        for i0 in range(0, q, 1024):
            i1 = min(q, i0 + 1024)
            z = torch.matmul(x[:, :, i0:i1].reshape(g, -1, d), k.transpose(-1, -2)).float().reshape(g, h // g, i1 - i0, n)
            z = z * s["scale"]
            if q > 1:
                seen = torch.arange(n, device=z.device) <= torch.arange(i0, i1, device=z.device)[:, None] + (n - q)
                z = z.masked_fill(~seen, float("-inf"))
            out[at + i0:at + i1] = torch.logsumexp(z, -1).permute(2, 0, 1).reshape(i1 - i0, h)
        at += q
    return out


def _prepare_norm(case, dev, gen):
    t, h, k = case["tokens"], case["heads"], case["size"]
    x = X_TYPES[case["type"]]
    s = {"case": case}
    if h > 1:
        # the fused projection's output: the heads, and as many values again beside them
        s["x"] = _heads(gen, dev, t, 2 * h, k, x, 0.4)
    else:
        s["x"] = (0.5 * _heads(gen, dev, t, 1, k, torch.float32, 0.3)).to(X_TYPES[case["in"]])
    if case["res"] != "none":
        # a residual stream: a few channels are much larger than the others
        s["r"] = _heads(gen, dev, t, 1, k, torch.float32, 1.0).to(X_TYPES[case["res"]])
        s["s"] = torch.empty_like(s["r"])
    w = 0.1 * torch.randn((k,), generator=gen, device=dev) + (1.0 - case["add"])
    s["w"] = w.to(x)
    s["y"] = torch.empty((t, h, k), dtype=x, device=dev)
    if case["out"] == "i8":
        s["codes"] = torch.empty((t, k), dtype=torch.int8, device=dev)
        s["a"] = torch.empty((t,), dtype=torch.float32, device=dev)
    return s


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * int(seed) + 29)
    if case["op"] == "norm":
        return _prepare_norm(case, dev, gen)
    n, g, page = case["seqs"], case["kv_heads"], case["page"]
    total = _lengths(case)
    per = -(-max(total) // page)
    pages = n * per + 5
    s = {"case": case, "per": per, "pages": pages, "total": total}
    order = torch.randperm(pages, generator=gen, device=dev)
    s["table"] = order[:n * per].to(torch.int32).reshape(n, per)
    s["lens"] = torch.tensor(total, dtype=torch.int32, device=dev)
    shape = (pages, g, page)
    # weights received in some steps so far: few tokens have much, some have none at all
    w = torch.exp(1.5 * torch.randn(shape, generator=gen, device=dev)) * (4.0 / max(total))
    s["weight"] = torch.where(torch.rand(shape, generator=gen, device=dev) < 0.05, torch.zeros_like(w), w)
    if case["op"] == "keep":
        s["keep"] = torch.empty((n, g, case["budget"]), dtype=torch.int32, device=dev)
        s["new_lens"] = torch.empty((n,), dtype=torch.int32, device=dev)
        return s
    d, x = case["dim"], X_TYPES[case["type"]]
    for name, spread in (("k", 0.4), ("v", 0.2)):
        if name == "v" and case["op"] == "weights":
            continue
        c = _heads(gen, dev, pages * page, g, d, x, spread).reshape(pages, page, g, d).transpose(1, 2)
        if case["kv"] == "x16":
            s[name + "_cache"], s[name + "_scale"] = c.contiguous(), None
        else:
            s[name + "_cache"], s[name + "_scale"] = (y.contiguous() for y in _quantised(c, case["kv"]))
        del c
    if case["op"] == "compact":
        # for each head the first and the newest tokens, and others between them
        at = torch.arange(per * page, device=dev)
        length = s["lens"][:, None, None]
        rank = torch.rand((n, g, per * page), generator=gen, device=dev)
        rank = torch.where((at < case["first"]) | (at >= length - case["recent"]), rank + 1.0, rank)
        rank = torch.where(at < length, rank, rank - 2.0)
        pick = rank.argsort(-1, descending=True)[..., :case["budget"]]
        pick = torch.where(pick < length, pick, torch.full_like(pick, per * page)).sort(-1).values
        keep = torch.full((n, g, case["budget"]), -1, dtype=torch.int32, device=dev)
        keep[..., :pick.shape[-1]] = torch.where(pick < length, pick, torch.full_like(pick, -1)).to(torch.int32)
        s["keep"] = keep
        to_per = -(-case["budget"] // page)
        if case["to"] == "same":
            s["to"], s["to_per"] = None, 0
        else:
            # pages of their own, behind those of the sequences
            more = n * to_per
            for name in ("k_cache", "v_cache", "k_scale", "v_scale", "weight"):
                if s[name] is not None:
                    old = s[name]
                    s[name] = torch.zeros((pages + more, *old.shape[1:]), dtype=old.dtype, device=dev)
                    _raw(s[name])[:pages] = _raw(old)
            s["to"] = (pages + torch.randperm(more, generator=gen, device=dev)).to(torch.int32).reshape(n, to_per)
            s["to_per"] = to_per
            s["pages"] = pages + more
        return s
    s["new"] = _rows(case)
    s["scale"] = _scale(d)
    s["q"] = _heads(gen, dev, sum(s["new"]), case["q_heads"], d, x, 0.4)
    cu = [0]
    for q in s["new"]:
        cu.append(cu[-1] + q)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    # the newest tokens have no weight yet
    s["known"] = torch.tensor([t - q for t, q in zip(total, s["new"])], dtype=torch.int32, device=dev)
    s["lse"] = _lse(s)
    return s


# --------------------------------------------------------------- plain forms

def _plain_norm(s):
    case = s["case"]
    x = s["x"][:, :case["heads"]].float()
    if case["res"] != "none":
        x = x + s["r"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (s["w"].float() + case["add"])
    out = {} if case["res"] == "none" else {"s": x.to(s["r"].dtype)}
    if case["out"] == "i8":
        y = y[:, 0]
        most = y.abs().amax(-1, keepdim=True)
        code = torch.round(y * torch.where(most > 0, 127.0 / most, torch.zeros_like(most)))
        out["y"] = (code * (most / 127.0)).to(s["w"].dtype)
    else:
        out["y"] = y.to(s["w"].dtype)
    return out


def _plain_weights(s):
    case = s["case"]
    h, g, d, n, page = case["q_heads"], case["kv_heads"], case["dim"], case["seqs"], case["page"]
    dev, most, l = s["q"].device, max(s["new"]), s["per"] * page
    table = s["table"].long()
    cu, length, known = s["cu"].long(), s["lens"].long(), s["known"].long()
    # query rows by sequence, each row's heads that share a key/value head beside one another
    i = torch.arange(most, device=dev)
    there = i < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + i).clamp_(max=max(0, s["q"].shape[0] - 1))
    q = s["q"][rows].float().reshape(n, most, g, h // g, d).permute(0, 2, 1, 3, 4).reshape(n, g, -1, d)
    lse = s["lse"][rows].reshape(n, most, g, h // g).permute(0, 2, 1, 3)
    p = torch.matmul(q, _cached(s["k_cache"], s["k_scale"], table).transpose(-1, -2)).reshape(n, g, most, h // g, l)
    p = p.mul_(s["scale"]).sub_(lse[..., None]).exp_()
    j = torch.arange(l, device=dev)
    last = i + (length - (cu[1:] - cu[:-1]))[:, None]
    seen = there[:, :, None] & (j <= last[..., None]) & (j < length[:, None, None])
    add = p.masked_fill_(~seen[:, None, :, None, :], 0.0).sum((2, 3))
    # add to the cells of the tokens that the sequence has
    seq = torch.arange(n, device=dev)[:, None].expand(n, l)
    j = j.expand(n, l)
    has = (j < length[:, None]) & (cu[1:] > cu[:-1])[:, None]
    seq, j = seq[has], j[has]
    at, row = table[seq, j // page], j % page
    old = torch.where((j < known[seq])[:, None], s["weight"][at, :, row] * case["decay"], torch.zeros((), device=dev))
    s["weight"][at, :, row] = old + add[seq, :, j]
    return {"weight": s["weight"]}


def _plain_keep(s):
    case = s["case"]
    n, g, page, budget, first, recent = (case[k] for k in ("seqs", "kv_heads", "page", "budget", "first", "recent"))
    l = s["per"] * page
    w = s["weight"][s["table"].long()].transpose(1, 2).reshape(n, g, l)
    j, length = torch.arange(l, device=w.device), s["lens"].long()[:, None, None]
    w = torch.where((j < first) | (j >= length - recent), torch.full_like(w, float("inf")), w)
    w = torch.where(j < length, w, torch.full_like(w, float("-inf")))
    pick = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    pick = torch.where(pick < length, pick, torch.full_like(pick, l)).sort(-1).values
    keep = torch.full((n, g, budget), -1, dtype=torch.int32, device=w.device)
    keep[..., :pick.shape[-1]] = torch.where(pick < l, pick, torch.full_like(pick, -1)).to(torch.int32)
    return {"keep": keep, "lens": s["lens"].clamp(max=budget)}


def _plain_compact(s):
    case = s["case"]
    page = case["page"]
    b, head, to = torch.nonzero(s["keep"] >= 0, as_tuple=True)
    source = s["keep"][b, head, to].long()
    table = s["table"].long()
    onto = table if s["to"] is None else s["to"].long()
    from_page, to_page = table[b, source // page], onto[b, to // page]
    out = {}
    for name in ("k_cache", "v_cache", "k_scale", "v_scale", "weight"):
        if s[name] is not None:
            c = _raw(s[name])
            c[to_page, head, to % page] = c[from_page, head, source % page]
            out[name] = s[name]
    return out


# ------------------------------------------------------ the framework's calls

def _own_norm(s, tb):
    case = s["case"]
    types = {"f32": tb.TERN_OUT_F32, "bf16": tb.TERN_OUT_BF16, "f16": tb.TERN_OUT_F16}
    x = tb.TERN_X_BF16 if case["type"] == "bf16" else tb.TERN_X_F16
    t, h, k = case["tokens"], case["heads"], case["size"]
    ldx = k if h == 1 else 2 * h * k
    if case["res"] == "none":
        out, res = {}, (tb.TERN_OUT_F32, None, 0, None, 0)
    else:
        out, res = {"s": s["s"]}, (types[case["res"]], s["r"], k, s["s"], k)
    if case["out"] == "i8":
        tb.tern_rms_norm_i8(x, types[case["in"]], t, k, s["x"], ldx, *res, s["w"], case["add"], EPS, s["codes"], s["a"])
        # what the codes stand for: the even, then the odd ones of each 16 values lie together
        codes = s["codes"].view(t, k // 16, 2, 8).transpose(2, 3)
        torch.mul(codes, s["a"][:, None, None, None], out=s["y"].view(t, k // 16, 8, 2))
        out["y"] = s["y"][:, 0]
    else:
        tb.tern_rms_norm(x, types[case["in"]], t, h, k, s["x"], ldx, *res, s["w"], case["add"], EPS, s["y"], h * k)
        out["y"] = s["y"]
    return out


def _own(s):
    from ternary_bit_weight_gb300 import binding as tb
    case = s["case"]
    if case["op"] == "norm":
        return _own_norm(s, tb)
    n, g, page = case["seqs"], case["kv_heads"], case["page"]
    if case["op"] == "keep":
        tb.tern_kv_keep(n, g, s["pages"], page, s["weight"], s["table"], s["per"], s["lens"], case["budget"], case["first"],
                        case["recent"], s["keep"], s["new_lens"])
        return {"keep": s["keep"], "lens": s["new_lens"]}
    kv = {"x16": tb.TERN_KV_X16, "e4m3": tb.TERN_KV_E4M3, "i8": tb.TERN_KV_I8}[case["kv"]]
    d = case["dim"]
    if case["op"] == "compact":
        tb.tern_kv_compact(kv, n, g, d, s["pages"], page, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["weight"],
                           s["table"], s["per"], s["keep"], case["budget"], s["to"], s["to_per"])
        return {k: s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale", "weight") if s[k] is not None}
    x, h = tb.TERN_X_BF16 if case["type"] == "bf16" else tb.TERN_X_F16, case["q_heads"]
    tb.tern_attn_weights(x, kv, n, s["cu"], s["q"].shape[0], h, g, d, s["scale"], s["q"], h * d, s["lse"], s["pages"], page,
                         s["k_cache"], s["k_scale"], s["table"], s["per"], s["lens"], s["known"], case["decay"], s["weight"])
    return {"weight": s["weight"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"norm": _plain_norm, "weights": _plain_weights, "keep": _plain_keep, "compact": _plain_compact}[op](state)


# ------------------------------------------------------------------- 64 bits

def _exact_norm(s):
    case = s["case"]
    x = s["x"][:, :case["heads"]].double()
    if "r" in s:
        x = x + s["r"].double()
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["size"] + EPS) * (s["w"].double() + case["add"])
    out = {"s": x} if "r" in s else {}
    if case["out"] == "i8":
        y = y[:, 0]
        step = y.abs().amax(-1, keepdim=True) / 127.0
        y = torch.round(y / step.clamp(min=1e-300)) * step
    return out | {"y": y}


def _exact_weights(s):
    case = s["case"]
    h, g, page = case["q_heads"], case["kv_heads"], case["page"]
    weight = s["weight"].double()
    at = 0
    for b, (q, n) in enumerate(zip(s["new"], s["total"])):
        if q == 0 or n == 0:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        k = _raw(s["k_cache"])[pages].view(s["k_cache"].dtype).double()
        if s["k_scale"] is not None:
            k = k * s["k_scale"][pages].double()[..., None]
        k = k.transpose(0, 1).reshape(g, -1, k.shape[-1])[:, :n]
        add = torch.zeros((g, n), dtype=torch.float64, device=k.device)
        for head in range(h):
            for i0 in range(0, q, 512):
                i1 = min(q, i0 + 512)
                z = s["q"][at + i0:at + i1, head].double() @ k[head // (h // g)].T * s["scale"]
                e = torch.exp(z - s["lse"][at + i0:at + i1, head].double()[:, None])
                add[head // (h // g)] += torch.tril(e, n - q + i0).sum(0)
        at += q
        new = torch.zeros((g, len(pages) * page), dtype=torch.float64, device=k.device)
        new[:, :n] = add
        j = torch.arange(len(pages) * page, device=k.device)
        old = weight[pages].transpose(0, 1).reshape(g, -1)
        new += torch.where(j < n - q, old * case["decay"], torch.zeros_like(old))
        new = torch.where(j < n, new, old)
        weight[pages] = new.reshape(g, len(pages), page).transpose(0, 1)
    return {"weight": weight}


def _exact_compact(s):
    """The lists one by one, with slots of the flattened cache."""
    case = s["case"]
    g, page = case["kv_heads"], case["page"]
    keep, table = s["keep"].cpu().numpy(), s["table"].cpu().numpy().astype(np.int64)
    onto = table if s["to"] is None else s["to"].cpu().numpy().astype(np.int64)
    source, target = [], []
    for b in range(case["seqs"]):
        for head in range(g):
            src = keep[b, head][keep[b, head] >= 0].astype(np.int64)
            dst = np.arange(len(src), dtype=np.int64)
            source.append((table[b][src // page] * g + head) * page + src % page)
            target.append((onto[b][dst // page] * g + head) * page + dst % page)
    source, target = (torch.from_numpy(np.concatenate(x)).to(s["keep"].device) for x in (source, target))
    out = {}
    for name in ("k_cache", "v_cache", "k_scale", "v_scale", "weight"):
        if s[name] is None:
            continue
        if s[name].dtype == torch.int8:     # codes: whole numbers
            out[name] = None
            continue
        c = s[name].double()
        flat = c.view(-1, c.shape[-1]) if c.dim() == 4 else c.view(-1)
        flat[target] = flat[source]
        out[name] = c
    return out


def exact(case, seed):
    if case["op"] == "keep":
        return None     # whole numbers alone
    s = prepare(case, seed)
    return {"norm": _exact_norm, "weights": _exact_weights, "compact": _exact_compact}[case["op"]](s)
