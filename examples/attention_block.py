"""The attention block of one 27B-class decoder layer (5120 -> 40 query heads and
8 key/value heads of dimension 128), run as a server runs it: prompts in parts,
then decoding steps, with ternary projections and an 8-bit paged cache.

  qkv = tern_linear_ex(x)                       ternary projection, bf16 out
  q, cache <- tern_rope_kv_write(qkv)           rotate, quantise, store
  part of a prompt:  k, v = tern_kv_read(cache) everything so far, then
                     o = tern_attn_prompt(q, k, v)
  decoding step:     o = tern_attn_decode(q, cache)
  y = tern_linear_ex(o)                         ternary projection

Every step runs on the GPU through libtern; the script prints the times and
compares the last decoding step with the same block computed from the formulas
in 64 bits (--check, on by default).

    python examples/attention_block.py [--seqs 4] [--prompt 1500] [--part 512] [--steps 8] [--cache e4m3]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import synth  # noqa: E402
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402

HQ, HKV, D, HIDDEN = 40, 8, 128, 5120
PAGE = 16
SCALE = D ** -0.5


class Linear:
    """A ternary projection in the GPU tile layout, bf16 in and out."""

    def __init__(self, name, dev):
        wl = synth.WORKLOADS["dec27b"]
        lin = next(l for l in wl.linears if l.name == name)
        self.N, self.K = lin.N, lin.K
        t, s = synth.weights(wl, 0, lin)
        t = torch.from_numpy(t).to(dev)
        packed = torch.empty((self.N, self.K // 4), dtype=torch.uint8, device=dev)
        tb.tern_pack(t, self.N, self.K, packed)
        scales = torch.from_numpy(s.view("int16")).to(dev)
        self.tiled = torch.empty(tb.tern_tiled_bytes(self.N, self.K), dtype=torch.uint8, device=dev)
        tb.tern_repack(packed, scales, self.N, self.K, self.tiled)
        self.dense = t.double() * scales.view(torch.float16).double().repeat_interleave(128, 1)   # for the check only
        self.ws = {}

    def __call__(self, x):
        m = x.shape[0]
        if m not in self.ws:
            self.ws[m] = torch.zeros(tb.tern_workspace_bytes(m, self.N, self.K), dtype=torch.uint8, device=x.device)
        y = torch.empty((m, self.N), dtype=torch.bfloat16, device=x.device)
        tb.tern_linear_ex(x, tb.TERN_X_BF16, self.K, self.tiled, m, self.K, [self.N], [y], [self.N], tb.TERN_OUT_BF16,
                          self.ws[m])
        return y


class Cache:
    """A paged cache of `seqs` sequences, pages dealt out in order of need."""

    def __init__(self, kind, seqs, longest, dev):
        self.kind = {"x16": tb.TERN_KV_X16, "e4m3": tb.TERN_KV_E4M3, "i8": tb.TERN_KV_I8}[kind]
        self.per = -(-longest // PAGE)
        self.pages = seqs * self.per
        shape = (self.pages, HKV, PAGE, D)
        dtype = torch.bfloat16 if kind == "x16" else torch.uint8
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device=dev) for _ in range(2))
        self.ks, self.vs = (None if kind == "x16" else torch.zeros(shape[:3], device=dev) for _ in range(2))
        order = torch.randperm(self.pages, generator=torch.Generator().manual_seed(0))
        self.table = order.to(torch.int32).reshape(seqs, self.per).to(dev)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device=dev)

    def slots(self, seq, position):
        """Slots of tokens at `position` [n] of sequences `seq` [n]."""
        return self.table[seq, position // PAGE].long() * PAGE + position % PAGE

    @property
    def arguments(self):
        return self.pages, PAGE, self.k, self.v, self.ks, self.vs


class Block:
    def __init__(self, kind, seqs, longest, dev):
        self.qkv, self.o = Linear("qkv", dev), Linear("o", dev)
        self.cache = Cache(kind, seqs, longest, dev)
        freq, self.amplitude = tb.tern_rope_freqs(D, 1e6, tb.TERN_ROPE_SCALE_PARTS, 4.0, 8192.0)
        self.freq = torch.tensor(freq, dtype=torch.float32, device=dev)
        self.ws_decode = torch.zeros(tb.tern_attn_decode_workspace_bytes(seqs, HQ, HKV, D, self.cache.per * PAGE),
                                     dtype=torch.uint8, device=dev)

    def store(self, qkv, seq, position):
        """Rotated queries; the keys and values go to the cache."""
        t, ld = qkv.shape
        q = torch.empty((t, HQ * D), dtype=qkv.dtype, device=qkv.device)
        tb.tern_rope_kv_write(tb.TERN_X_BF16, self.cache.kind, tb.TERN_ROPE_HALF, t, HQ, HKV, D, D,
                              position.to(torch.int32), self.freq, self.amplitude, qkv, ld, q, HQ * D,
                              qkv[:, HQ * D:], ld, qkv[:, (HQ + HKV) * D:], ld, self.cache.slots(seq, position),
                              *self.cache.arguments)
        return q

    def prompt_part(self, x, new):
        """x [seqs * new, hidden]: the next `new` tokens of every prompt, packed."""
        dev, c = x.device, self.cache
        seqs = c.lens.numel()
        past = int(c.lens[0])                      # prompts of one length here
        seq = torch.arange(seqs, device=dev).repeat_interleave(new)
        q = self.store(self.qkv(x), seq, past + torch.arange(new, device=dev).repeat(seqs))
        c.lens += new
        total = past + new
        # all keys and values so far, packed by sequence
        rows = seqs * total
        k, v = (torch.empty((rows, HKV * D), dtype=x.dtype, device=dev) for _ in range(2))
        everything = c.slots(torch.arange(seqs, device=dev).repeat_interleave(total), torch.arange(total, device=dev).repeat(seqs))
        tb.tern_kv_read(tb.TERN_X_BF16, c.kind, rows, HKV, D, everything, *c.arguments, k, HKV * D, v, HKV * D)
        o = torch.empty((x.shape[0], HQ * D), dtype=x.dtype, device=dev)
        cu = torch.arange(seqs + 1, dtype=torch.int32, device=dev)
        ws = torch.zeros(tb.tern_attn_prompt_workspace_bytes(seqs, x.shape[0], rows, HQ, HKV, D), dtype=torch.uint8, device=dev)
        tb.tern_attn_prompt(tb.TERN_X_BF16, seqs, cu * new, cu * total, x.shape[0], rows, HQ, HKV, D, True, SCALE,
                            q, HQ * D, k, HKV * D, v, HKV * D, o, HQ * D, None, ws)
        return self.o(o)

    def step(self, x):
        """x [seqs, hidden]: one new token of every sequence."""
        c = self.cache
        q = self.store(self.qkv(x), torch.arange(c.lens.numel(), device=x.device), c.lens.long())
        c.lens += 1
        o = torch.empty((x.shape[0], HQ * D), dtype=x.dtype, device=x.device)
        tb.tern_attn_decode(tb.TERN_X_BF16, c.kind, x.shape[0], HQ, HKV, D, SCALE, q, HQ * D, *c.arguments, c.table, c.per,
                            c.lens, o, HQ * D, None, self.ws_decode)
        return self.o(o)


def reference(block, xs):
    """The last token's output of every sequence in 64 bits, nothing rounded: xs [seqs, tokens, hidden]."""
    seqs, n, _ = xs.shape
    qkv = xs.double() @ block.qkv.dense.T
    angle = torch.arange(n, device=xs.device).double()[:, None] * block.freq.double()
    c, s = angle.cos()[:, None] * block.amplitude, angle.sin()[:, None] * block.amplitude
    heads = qkv.reshape(seqs, n, HQ + 2 * HKV, D)
    a, b = heads[:, :, :HQ + HKV, :D // 2], heads[:, :, :HQ + HKV, D // 2:]
    rotated = torch.cat([a * c - b * s, b * c + a * s], -1)
    q, k, v = rotated[:, -1, :HQ], rotated[:, :, HQ:], heads[:, :, HQ + HKV:]
    q = q.reshape(seqs, HKV, HQ // HKV, D)
    p = torch.softmax(torch.einsum("bgrd,bngd->bgrn", q, k) * SCALE, -1)
    o = torch.einsum("bgrn,bngd->bgrd", p, v).reshape(seqs, HQ * D)
    return o @ block.o.dense.T


def run(seqs=4, prompt=1500, part=512, steps=8, cache="e4m3", check=True, out=print):
    dev = torch.device("cuda:0")
    block = Block(cache, seqs, prompt + steps, dev)
    gen = torch.Generator(device=dev).manual_seed(1)
    xs = torch.randn((seqs, prompt + steps, HIDDEN), generator=gen, device=dev).to(torch.bfloat16)

    def timed(f, *args):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        y = f(*args)
        b.record()
        torch.cuda.synchronize()
        return y, a.elapsed_time(b) * 1e3

    at = 0
    while at < prompt:
        new = min(part, prompt - at)
        _, us = timed(block.prompt_part, xs[:, at:at + new].reshape(-1, HIDDEN).contiguous(), new)
        out(f"prompt tokens {at}..{at + new - 1} of {seqs} sequences: {us:.0f} us")
        at += new
    for i in range(steps):
        y, us = timed(block.step, xs[:, at + i].contiguous())
        out(f"decoding step {i}: {us:.0f} us")
    err = None
    if check:
        want = reference(block, xs)
        err = float((y.double() - want).norm() / want.norm())
        out(f"last step against 64 bits: relative error {err:.4f}")
    return err


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=1500)
    ap.add_argument("--part", type=int, default=512)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--cache", choices=["x16", "e4m3", "i8"], default="e4m3")
    ap.add_argument("--no-check", dest="check", action="store_false")
    a = ap.parse_args()
    run(a.seqs, a.prompt, a.part, a.steps, a.cache, a.check)
