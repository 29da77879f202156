"""Accumulated attention weights where every loop of the kernels turns: more tiles than warps,
more items than CTAs, more sequences than a warp has lanes, idle ones among them.

The caches are made on the GPU and the 64-bit reference is one product per head, so that the
sizes can be those at which a warp refills its ring and changes from one batch of tiles to the
next.  Bounds as in test_gpu_attn_weights.py.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import TYPES  # noqa: E402
from budget_util import KV, X16  # noqa: E402
from gpu_util import DEV  # noqa: E402
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402

pytestmark = pytest.mark.gpu


class Case:
    """`rows[b]` newest of `lens[b]` tokens as query rows, everything on the GPU."""

    def __init__(self, seed, lens, rows, Hq, Hkv, D, page, kv, t):
        self.lens, self.rows, self.Hq, self.Hkv, self.D, self.page, self.kv, self.t = lens, rows, Hq, Hkv, D, page, kv, t
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.per = -(-max(lens) // page)
        used = [-(-n // page) for n in lens]
        self.pages = sum(used) + 2
        order = torch.randperm(self.pages, generator=g, device=DEV).to(torch.int32)
        self.table = torch.full((len(lens), self.per), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.pages, Hkv, page)
        size = torch.exp(0.4 * torch.randn((1, Hkv, 1, D), generator=g, device=DEV))
        if kv == "x16":
            self.k = (torch.randn((*shape, D), generator=g, device=DEV) * size).to(TYPES[t])
            self.ks = None
        else:
            self.ks = torch.exp(0.3 * torch.randn(shape, generator=g, device=DEV)) / (60.0 if kv == "i8" else 200.0)
            if kv == "i8":
                self.k = torch.randint(-127, 128, (*shape, D), generator=g, device=DEV, dtype=torch.int8)
            else:
                self.k = (120.0 * torch.randn((*shape, D), generator=g, device=DEV)).clamp(-448, 448).to(torch.float8_e4m3fn)
        self.weight = torch.rand(shape, generator=g, device=DEV)
        cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
        self.cu = cu
        self.q = (torch.randn((cu[-1], Hq * D), generator=g, device=DEV) *
                  torch.exp(0.4 * torch.randn((1, Hq * D), generator=g, device=DEV))).to(TYPES[t])
        self.scale = float(np.float32(D ** -0.5))
        self.dev_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.dev_cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        self.known = [max(0, n - r - b % 3) for b, (n, r) in enumerate(zip(lens, rows))]
        self.dev_known = torch.tensor(self.known, dtype=torch.int32, device=DEV)
        self.lse = torch.full((cu[-1], Hq), float("-inf"), dtype=torch.float32, device=DEV)

    def keys(self, b):
        """[Hkv, n, D] in 64 bits, and where the tokens lie."""
        j = torch.arange(self.lens[b], device=DEV)
        page, row = self.table[b].long()[j // self.page], j % self.page
        k = self.k.view(torch.uint8) if self.kv != "x16" else self.k
        k = k[page, :, row].view(self.k.dtype).double().transpose(0, 1)
        if self.ks is not None:
            k = k * self.ks[page, :, row].T.double()[..., None]
        return k, page, row

    def reference(self, decay):
        """Fills the logarithms; (weights, bound) of the whole plane in 64 bits."""
        G, D = self.Hq // self.Hkv, self.D
        want, bound = self.weight.double(), torch.zeros_like(self.weight, dtype=torch.float64)
        for b, n in enumerate(self.lens):
            q0, nq = self.cu[b], self.rows[b]
            if n == 0 or nq == 0:
                continue
            k, page, row = self.keys(b)
            j = torch.arange(n, device=DEV)
            seen = j <= torch.arange(nq, device=DEV)[:, None] + n - nq
            x = self.q[q0:q0 + nq].double().reshape(nq, self.Hq, D)
            add, err = (torch.zeros((self.Hkv, n), dtype=torch.float64, device=DEV) for _ in range(2))
            for h in range(self.Hq):
                kk = k[h // G]
                s, S = x[:, h] @ kk.T * self.scale, x[:, h].abs() @ kk.abs().T * self.scale
                l = torch.logsumexp(s.masked_fill(~seen, float("-inf")), 1).float()
                self.lse[q0:q0 + nq, h] = l
                l = l.double()[:, None]
                p = torch.exp(s - l).masked_fill(~seen, 0.0)
                e = D * 2.0 ** -23 * S + 2.0 ** -21 * S + 2.0 ** -23 * l.abs() + 2.0 ** -20
                add[h // G] += p.sum(0)
                err[h // G] += (p * e * (1 + e)).sum(0)
            old = self.weight.double()[page, :, row].T
            new = torch.where(j < self.known[b], decay * old, 0.0) + add
            terms = nq * G
            want[page, :, row] = new.T
            bound[page, :, row] = (err + terms * 2.0 ** -24 * add + terms * 2.0 ** -126 + 2.0 ** -23 * new).T
        return want, bound

    def run(self, decay, single=False, known=True):
        w = self.weight.clone()
        tb.tern_attn_weights(X16[self.t], KV[self.kv], len(self.lens), None if single else self.dev_cu, self.cu[-1], self.Hq,
                             self.Hkv, self.D, self.scale, self.q, self.Hq * self.D, self.lse, self.pages, self.page, self.k,
                             self.ks, self.table, self.per, self.dev_lens, self.dev_known if known else None, decay, w)
        return w

    def check(self, decay=0.75, single=False):
        want, bound = self.reference(decay)
        got = self.run(decay, single)
        bad = ~((got.double() - want).abs() <= bound)
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}: " \
                              f"{float(got[bad][0])} {float(want[bad][0])} {float(bound[bad][0])}"
        for _ in range(2):
            assert torch.equal(self.run(decay, single), got)


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def ragged(seed, n, longest, idle):
    """n lengths spread over a factor of sixteen, every `idle`-th one zero."""
    g = np.random.RandomState(seed)
    lens = np.exp(g.uniform(np.log(longest / 16), np.log(longest), n)).astype(int)
    lens[n // 2] = longest
    lens[3::idle] = 0
    return lens.tolist()


@pytest.mark.parametrize("kv,t,Hq,Hkv,D", [("x16", "bf16", 40, 8, 128), ("x16", "f16", 16, 16, 64), ("e4m3", "bf16", 32, 16, 128),
                                           ("i8", "f16", 16, 16, 128), ("i8", "bf16", 64, 16, 64), ("x16", "bf16", 96, 8, 64),
                                           ("e4m3", "bf16", 72, 8, 96), ("i8", "bf16", 128, 8, 128)])
def test_many_tiles_to_a_warp(kv, t, Hq, Hkv, D):
    """More than 40 tiles of 32 keys for each warp that an SM can hold (up to 16): rings are refilled, batches of 32 tiles
    follow one another, and a warp goes on from sequence to sequence and head to head; up to 8 heads to a group and more."""
    two = 32 * D * (2 if kv == "x16" else 1) <= 4096 and Hq // Hkv <= 8
    longest = 8192
    lens = ragged(D + Hq, 70, longest, 11)
    while sum(-(-n // 32) for n in lens) * Hkv < 42 * sms() * (16 if two else 8):
        lens += ragged(len(lens), 35, longest, 9)
    c = Case(Hq + D, lens, [1 if n else 0 for n in lens], Hq, Hkv, D, 32, kv, t)
    c.check()


@pytest.mark.parametrize("kv,D", [("x16", 64), ("i8", 128)])
def test_many_tiles_of_one_row_each(kv, D):
    """Without offsets, everything known: row b is sequence b's, whether it has tokens or not."""
    lens = ragged(D, 150, 6000, 7)
    c = Case(D, lens, [1] * 150, 8, 8, D, 64, kv, "bf16")
    c.known = lens
    c.dev_known = c.dev_lens
    c.check(single=True)
    assert torch.equal(c.run(0.75, True, known=False), c.run(0.75, True))


@pytest.mark.parametrize("page,kv,D,Hq,Hkv", [(4, "x16", 128, 10, 2), (8, "i8", 64, 8, 8), (1, "e4m3", 80, 12, 4)])
def test_many_items_of_small_pages(page, kv, D, Hq, Hkv):
    """More runs of keys than warps, over several groups of 32 sequences."""
    lens = ragged(page, 70, 4000, 9)
    keys = 8192 // ((128 if D > 64 else 64) * (2 if kv == "x16" else 1))
    while sum(-(-n // keys) for n in lens) * Hkv < 3 * sms() * 16:
        lens += ragged(len(lens), 70, 4000, 9)
    Case(page + D, lens, [min(n, 1 + b % 2) for b, n in enumerate(lens)], Hq, Hkv, D, page, kv, "bf16").check()


@pytest.mark.parametrize("kv,t,Hq,Hkv,D", [("x16", "bf16", 40, 8, 128), ("e4m3", "bf16", 16, 8, 128), ("i8", "bf16", 40, 8, 64),
                                           ("x16", "f16", 24, 8, 80), ("i8", "f16", 12, 4, 128), ("e4m3", "f16", 16, 16, 64)])
def test_many_items_to_a_cta(kv, t, Hq, Hkv, D):
    """Windows and whole prompts: three blocks of 128 keys and more for each CTA, odd and even numbers of them, over more
    than 32 sequences, some idle and some without rows."""
    lens = ragged(D + Hkv, 44, 1500, 7)
    while sum(-(-n // 128) for n in lens) * Hkv < 7 * sms():
        lens += ragged(len(lens), 20, 1500, 6)
    rows = [(0, 32, n, 1, 100, n // 2, 33)[b % 7] for b, n in enumerate(lens)]
    c = Case(D + Hq, lens, [min(r, n) for r, n in zip(rows, lens)], Hq, Hkv, D, 16, kv, t)
    assert c.cu[-1] * (Hq // Hkv) > 16 * len(lens)          # the form for many rows
    c.check()


@pytest.mark.parametrize("kv", ["x16", "i8"])
@pytest.mark.parametrize("seqs,chunk", [(64, 512), (128, 200), (300, 400)])
def test_decoding_steps_beside_a_chunk(kv, seqs, chunk):
    """Single tokens and one part of a prompt in one call; by their numbers in either form."""
    lens = ragged(seqs, seqs, 900, 13) + [chunk + 700] + [40] * 3
    rows = [min(1, n) for n in lens]
    rows[seqs] = chunk
    Case(seqs, lens, rows, 40, 8, 128, 16, kv, "bf16").check()
