"""A paged cache with a plane of weights, and the 64-bit references of the calls
that keep it within a budget."""
import numpy as np
import torch

from attn_util import TYPES, code_values, f64, quantise, randn
from gpu_util import DEV
from ternary_bit_weight_gb300 import binding as tb

X16 = {"bf16": tb.TERN_X_BF16, "f16": tb.TERN_X_F16}
KV = {"x16": tb.TERN_KV_X16, "e4m3": tb.TERN_KV_E4M3, "i8": tb.TERN_KV_I8}


class Cache:
    """`lens` tokens of each sequence in pages dealt at random, all of `pages` filled."""

    def __init__(self, seed, lens, Hkv, D, page, kv, t="bf16", per=None, spare=3):
        self.lens, self.Hkv, self.D, self.page, self.kv, self.t = list(lens), Hkv, D, page, kv, t
        self.per = per or max(1, -(-max(lens) // page))
        self.pages = len(lens) * self.per + spare
        g = torch.Generator().manual_seed(seed)
        order = torch.randperm(self.pages, generator=g)
        self.table = order[:len(lens) * self.per].to(torch.int32).reshape(len(lens), self.per)
        shape = (self.pages, Hkv, page, D)
        self.k, self.v, self.ks, self.vs = [], [], None, None
        x = [randn(seed + 1 + i, *shape) * torch.exp(0.4 * randn(seed + 5 + i, 1, Hkv, 1, D)) for i in range(2)]
        if kv == "x16":
            self.k, self.v = (y.to(TYPES[t]).to(DEV) for y in x)
        else:
            (k, ks), (v, vs) = (quantise(y.to(TYPES[t]), kv) for y in x)
            self.k, self.v, self.ks, self.vs = k.to(DEV), v.to(DEV), ks.to(DEV), vs.to(DEV)
        self.weight = torch.exp(randn(seed + 11, *shape[:3])).to(DEV)
        self.dev_table, self.dev_lens = self.table.to(DEV), torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def slots(self, b):
        """(page, row) of each token that the table has room for."""
        j = np.arange(self.per * self.page)
        return self.table[b].numpy()[j // self.page], j % self.page

    def keys(self, b, head):
        """[room, D] in 64 bits."""
        page, row = self.slots(b)
        page = np.clip(page, 0, self.pages - 1)
        k = f64(self.k) if self.kv == "x16" else code_values(self.k.cpu(), self.kv) * f64(self.ks)[..., None]
        return k[page, head, row]

    def planes(self):
        return {n: getattr(self, n) for n in ("k", "v", "ks", "vs", "weight") if getattr(self, n) is not None}


def keep_reference(weight, n, budget, first, recent):
    """Ascending list of one head's tokens; weight [n] float32."""
    if n <= budget:
        return np.arange(n)
    j = np.arange(n)
    must = (j < first) | (j >= n - recent)
    # the largest first, of equal ones the earlier; NaN after all of them
    order = sorted(j[~must], key=lambda i: (np.isnan(weight[i]), -weight[i] if not np.isnan(weight[i]) else 0.0, i))
    return np.sort(np.concatenate([j[must], np.array(order[:budget - first - recent], dtype=int)]))
