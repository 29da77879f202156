"""64-bit references and error bounds for the attention-side tests.

Bounds.  u is the unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 fp16).

Attention: a score is a sum of D exact products in fp32, off by at most
D * 2^-23 * scale * sum_d |q_d k_d| (S below is the largest of these sums),
and the exponential and its argument add 2^-20, so each weight is off by a
relative e = 2 * (D * 2^-23 * S + 2^-20), the factor for numerator and
denominator; sums of n weights add n * 2^-24.  Weights are rounded to 16 bits
for the product with V (relative w, the unit roundoff of that type; for fp16
also 2^-24 of the largest weight where a weight is below fp16's normal range).
With A_d = sum_j p_j |v_jd| the output is therefore within
  u |o_d| + A_d (e + w + n 2^-24) + n 2^-24 max_j |v_jd| + 2^-24
of the exact one (the last term: fp16 subnormals), and the logarithm within
e + n 2^-24 + 2^-21 |lse|.
"""
import numpy as np
import torch

from gpu_util import DEV

UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def randn(seed, *shape):
    """Seeded normals on the CPU, fp32."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g)


def heads(seed, rows, H, D, t, pad=0, spread=0.5):
    """[rows, H*D + pad] of type t on the GPU (padding NaN): channels of unequal size."""
    x = randn(seed, rows, H * D) * torch.exp(spread * randn(seed + 1, 1, H * D))
    out = torch.full((rows, H * D + pad), float("nan"), dtype=TYPES[t])
    out[:, :H * D] = x.to(TYPES[t])
    return out.to(DEV)


def attend(q, k, v, scale, seen):
    """One head in 64 bits: q [n, D], k and v [m, D], seen [n, m] ->
    output, logarithm, and the pieces A, S of the bounds."""
    n, D = q.shape
    if k.shape[0] == 0:
        z = np.zeros((n, D))
        return z, np.full(n, -np.inf), z, np.zeros(n)
    s = np.where(seen, q @ k.T * scale, -np.inf)
    S = np.where(seen, np.abs(q) @ np.abs(k).T * abs(scale), 0.0).max(1)
    m = s.max(1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    some = l > 0
    p = np.where(some, p / np.where(some, l, 1.0), 0.0)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0]
    return p @ v, lse, p @ np.abs(v), S


def bounds(o, lse, A, S, v, D, t, weight_type):
    """(bound on the output [n, D], bound on the logarithm [n])."""
    n = v.shape[0]
    e = 2 * (D * 2.0 ** -23 * S + 2.0 ** -20)[:, None]
    vmax = np.abs(v).max(0)[None] if n else 0.0
    tail = n * 2.0 ** -24 * vmax if weight_type == "f16" else 0.0
    bo = UNIT[t] * np.abs(o) + A * (e + UNIT[weight_type] + n * 2.0 ** -24) + tail + 2.0 ** -24
    bl = e[:, 0] + n * 2.0 ** -24 + 2.0 ** -21 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return bo, bl


def f64(x):
    return x.detach().double().cpu().numpy()


def assert_close(got, want, bound, what):
    got = np.asarray(got, dtype=np.float64)
    inf = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), inf), f"{what}: rows that see nothing differ"
    err = np.where(inf, 0.0, np.abs(np.where(inf, 0.0, got) - np.where(inf, 0.0, want)))
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {i}: got {got[i]} "
                             f"want {want[i]} bound {np.broadcast_to(bound, got.shape)[i]}")


# ------------------------------------------------------------------- cache

def quantise(x, kind):
    """The cache's rule in fp32: x [..., D] float32 -> codes (int8 or raw e4m3 bytes), factors."""
    top = np.float32(448.0 if kind == "e4m3" else 127.0)
    x = x.float().cpu()
    m = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    inv = torch.where((m > 0) & ~bad, (torch.tensor(top) / m).clamp(max=torch.finfo(torch.float32).max), torch.zeros(()))
    y = torch.where(bad[..., None], torch.zeros(()), x * inv[..., None])
    if kind == "e4m3":
        code = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        code = torch.round(y).to(torch.int8).view(torch.uint8)
    return code, torch.where(bad, torch.full((), float("nan")), m / torch.tensor(top))


def code_values(code, kind):
    """Raw code bytes -> values as float64."""
    return f64(code.view(torch.float8_e4m3fn).float() if kind == "e4m3" else code.view(torch.int8))
