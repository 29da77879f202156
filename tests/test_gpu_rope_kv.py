"""Rotary positions and the paged cache against 64-bit / rule-exact
references.

Rotation bound: the angle is reduced in double to a fraction of a turn held
in fp32 (2^-25 turns, 2^-22.3 radians) and sine and cosine are fp32 (a few
2^-24), so a rotated element is within u |y| + amplitude (|a| + |b|) 2^-20 +
2^-25 of the exact one (the last term: fp16 subnormals).  Codes and factors of
the cache follow a rule of IEEE fp32 steps and are compared bit for bit."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import TYPES, UNIT, code_values, f64, heads, quantise, randn  # noqa: E402
from gpu_util import DEV  # noqa: E402
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402

pytestmark = pytest.mark.gpu

X = {"bf16": tb.TERN_X_BF16, "f16": tb.TERN_X_F16}
LAYOUT = {"half": tb.TERN_ROPE_HALF, "interleaved": tb.TERN_ROPE_INTERLEAVED}
KV = {"x16": tb.TERN_KV_X16, "e4m3": tb.TERN_KV_E4M3, "i8": tb.TERN_KV_I8}


def rotated(x, pos, freq, amplitude, rot, layout):
    """x [T, H, D] in 64 bits -> (rotated, the bound's fp32 part)."""
    angle = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(freq, dtype=np.float32).astype(np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y, b = x.copy(), np.zeros_like(x)
    lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a0, a1 = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = amplitude * (a0 * c - a1 * s), amplitude * (a1 * c + a0 * s)
    b[..., lo] = b[..., hi] = amplitude * (np.abs(a0) + np.abs(a1)) * 2.0 ** -20
    return y, b


def positions(seed, T, most=1 << 20):
    pos = torch.from_numpy(np.random.default_rng(seed).integers(0, most, T).astype(np.int32))
    pos[0] = 0
    pos[-1] = most - 1
    return pos


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,t", [(1, 40, 8, 128, 128, "bf16"), (5, 16, 8, 128, 64, "f16"),
                                             (7, 3, 1, 80, 48, "bf16"), (3, 5, 0, 256, 256, "f16"),
                                             (4, 70, 2, 144, 16, "bf16"), (33, 1, 1, 16, 16, "bf16"),
                                             (2, 2, 2, 64, 0, "f16")])
def test_rope(T, Hq, Hk, D, rot, t, layout):
    pad = 8
    Q, K = heads(T + D, T, Hq, D, t, pad), heads(T + D + 5, T, max(Hk, 1), D, t, pad)
    pos = positions(T + rot, T)
    freq, _ = tb.tern_rope_freqs(rot, 1e6) if rot else ([], 1.0)
    f = torch.tensor(freq if freq else [0.0], dtype=torch.float32, device=DEV)
    amp = 1.25
    Qo = torch.full((T, Hq * D + 2 * pad), 7.0, dtype=TYPES[t], device=DEV)
    Ko = torch.full((T, max(Hk, 1) * D), 7.0, dtype=TYPES[t], device=DEV)
    tb.tern_rope(X[t], LAYOUT[layout], T, D, rot, pos.to(DEV), f, amp, Hq, Q, Hq * D + pad, Qo, Hq * D + 2 * pad,
                 Hk, K if Hk else None, max(Hk, 1) * D + pad, Ko if Hk else None, max(Hk, 1) * D)
    for src, dst, H in ((Q, Qo, Hq), (K, Ko, Hk)):
        if H == 0:
            assert torch.all(dst == 7.0)
            continue
        x = f64(src)[:, :H * D].reshape(T, H, D)
        want, b = rotated(x, pos.numpy(), freq, np.float32(amp).astype(np.float64), rot, layout) if rot else (x, 0 * x)
        got = f64(dst)[:, :H * D].reshape(T, H, D)
        assert np.all(np.abs(got - want) <= UNIT[t] * np.abs(want) + b + 2.0 ** -25)
        assert np.array_equal(got[..., rot:], x[..., rot:])
    assert torch.all(Qo[:, Hq * D:] == 7.0)     # nothing past the heads is written


def test_rope_in_place_and_large_positions():
    T, H, D = 6, 4, 128
    Q = heads(3, T, H, D, "bf16")
    pos = torch.tensor([0, 1, -1, -70000, 2 ** 31 - 1, 16777217], dtype=torch.int32)
    freq, amp = tb.tern_rope_freqs(D, 1e4, tb.TERN_ROPE_SCALE_PARTS, 8.0, 4096.0)
    f = torch.tensor(freq, dtype=torch.float32, device=DEV)
    want, b = rotated(f64(Q).reshape(T, H, D), pos.numpy(), freq, float(np.float32(amp)), D, "half")
    tb.tern_rope(tb.TERN_X_BF16, tb.TERN_ROPE_HALF, T, D, D, pos.to(DEV), f, amp, H, Q, H * D, Q, H * D)
    assert np.all(np.abs(f64(Q).reshape(T, H, D) - want) <= UNIT["bf16"] * np.abs(want) + b + 2.0 ** -25)


def make_cache(pages, Hkv, page, D, kind, t):
    shape = (pages, Hkv, page, D)
    dtype = TYPES[t] if kind == "x16" else torch.uint8
    fill = 3.0 if kind == "x16" else 0xA5
    k, v = (torch.full(shape, fill, dtype=dtype, device=DEV) for _ in range(2))
    ks, vs = (torch.full(shape[:3], -5.0, device=DEV) for _ in range(2))
    return k, v, (None if kind == "x16" else ks), (None if kind == "x16" else vs)


def scatter_slots(seed, T, pages, page):
    return torch.from_numpy(np.random.default_rng(seed).permutation(pages * page)[:T].astype(np.int64))


CACHES = [(1, 8, 128, 16, "bf16"), (5, 8, 128, 1, "f16"), (37, 3, 80, 4, "bf16"), (130, 1, 64, 32, "f16"),
          (19, 9, 16, 128, "bf16"), (3, 70, 112, 64, "f16")]


@pytest.mark.parametrize("kind", ["x16", "e4m3", "i8"])
@pytest.mark.parametrize("T,Hkv,D,page,t", CACHES)
def test_kv_write_and_read(T, Hkv, D, page, t, kind):
    pages = -(-2 * T // page) + 1
    K, V = heads(T, T, Hkv, D, t, 8, 1.0), heads(T + 9, T, Hkv, D, t, 16, 1.0)
    K[0, :D] = 0.0                              # a head of zeros
    V[T - 1, :D] *= 2.0 ** -9                   # and one of small values
    slots = scatter_slots(T + D, T, pages, page)
    cache = make_cache(pages, Hkv, page, D, kind, t)
    before = [None if c is None else c.clone() for c in cache]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tb.tern_kv_write(X[t], KV[kind], T, Hkv, D, K, Hkv * D + 8, V, Hkv * D + 16, slots.to(DEV), pages, page, *cache, err)
    assert int(err) == 0
    at, row = slots // page, slots % page
    Ko, Vo = (torch.full((T, Hkv * D + 8), 9.0, dtype=TYPES[t], device=DEV) for _ in range(2))
    tb.tern_kv_read(X[t], KV[kind], T, Hkv, D, slots.to(DEV), pages, page, *cache, Ko, Hkv * D + 8, Vo, Hkv * D + 8)
    for src, c, scale, old, old_scale, back in ((K, cache[0], cache[2], before[0], before[2], Ko),
                                                (V, cache[1], cache[3], before[1], before[3], Vo)):
        x = src[:, :Hkv * D].reshape(T, Hkv, D).cpu()
        want = old.cpu()
        if kind == "x16":
            want[at, :, row] = x
            assert torch.equal(c.cpu().view(torch.int16), want.view(torch.int16))
            value = x
        else:
            code, factor = quantise(x, kind)
            want[at, :, row] = code
            want_scale = old_scale.cpu()
            want_scale[at, :, row] = factor
            assert torch.equal(c.cpu(), want)
            assert torch.equal(scale.cpu(), want_scale)
            value = (torch.from_numpy(code_values(code, kind)).float() * factor[..., None]).to(TYPES[t])
        assert torch.equal(back[:, :Hkv * D].cpu().reshape(T, Hkv, D), value)
        assert torch.all(back[:, Hkv * D:] == 9.0)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_kv_special_values(kind):
    """Non-finite heads read back as NaN and touch nothing else; tiny heads keep their codes in range."""
    T, Hkv, D, page = 5, 2, 32, 8
    K = heads(1, T, Hkv, D, "bf16")
    V = heads(2, T, Hkv, D, "bf16")
    K[1, 3] = float("nan")
    K[2, D] = float("inf")
    V[3, 2 * D - 1] = float("-inf")
    K[4, :D] = torch.linspace(-1, 1, D, device=DEV).to(torch.bfloat16) * 2.0 ** -130   # 448 / max overflows fp32
    cache = make_cache(2, Hkv, page, D, kind, "bf16")
    slots = torch.tensor([3, 9, 0, 15, 7], device=DEV)
    tb.tern_kv_write(tb.TERN_X_BF16, KV[kind], T, Hkv, D, K, Hkv * D, V, Hkv * D, slots, 2, page, *cache)
    Ko, Vo = torch.empty_like(K), torch.empty_like(V)
    tb.tern_kv_read(tb.TERN_X_BF16, KV[kind], T, Hkv, D, slots, 2, page, *cache, Ko, Hkv * D, Vo, Hkv * D)
    for src, out, bad in ((K, Ko, {(1, 0), (2, 1)}), (V, Vo, {(3, 1)})):
        x, y = src.reshape(T, Hkv, D).cpu(), out.reshape(T, Hkv, D).cpu()
        for i in range(T):
            for g in range(Hkv):
                if (i, g) in bad:
                    assert torch.isnan(y[i, g]).all()
                else:
                    code, factor = quantise(x[i, g], kind)
                    want = (torch.from_numpy(code_values(code, kind)).float() * factor).to(torch.bfloat16)
                    assert torch.equal(y[i, g], want), (i, g)


def test_kv_slots_outside():
    """Negative slots are padding, slots past the cache are counted; both read as zeros."""
    T, Hkv, D, page, pages = 6, 2, 64, 4, 3
    K, V = heads(4, T, Hkv, D, "f16"), heads(5, T, Hkv, D, "f16")
    slots = torch.tensor([-1, 5, 12, 11, 1 << 40, -(1 << 50)], device=DEV)
    cache = make_cache(pages, Hkv, page, D, "x16", "f16")
    want = cache[0].clone()
    want[1, :, 1] = K[1].reshape(Hkv, D)
    want[2, :, 3] = K[3].reshape(Hkv, D)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tb.tern_kv_write(tb.TERN_X_F16, tb.TERN_KV_X16, T, Hkv, D, K, Hkv * D, V, Hkv * D, slots, pages, page, *cache, err)
    assert int(err) == 2
    assert torch.equal(cache[0], want)
    Ko, Vo = torch.full_like(K, 5.0), torch.full_like(V, 5.0)
    tb.tern_kv_read(tb.TERN_X_F16, tb.TERN_KV_X16, T, Hkv, D, slots, pages, page, *cache, Ko, Hkv * D, Vo, Hkv * D)
    for i in range(T):
        inside = i in (1, 3)
        assert torch.equal(Ko[i], K[i] if inside else torch.zeros_like(K[i]))
        assert torch.equal(Vo[i], V[i] if inside else torch.zeros_like(V[i]))


def test_kv_offsets_past_32_bits():
    """Pages whose byte and element offsets pass 2^32."""
    Hkv, D, page = 8, 128, 64
    pages = (1 << 32) // (Hkv * D * page) + 3
    k = torch.zeros((pages, Hkv, page, D), dtype=torch.uint8, device=DEV)
    v = torch.zeros((pages, Hkv, page, D), dtype=torch.uint8, device=DEV)
    ks, vs = (torch.zeros((pages, Hkv, page), device=DEV) for _ in range(2))
    K, V = heads(6, 2, Hkv, D, "bf16"), heads(7, 2, Hkv, D, "bf16")
    slots = torch.tensor([pages * page - 1, 3], device=DEV)
    tb.tern_kv_write(tb.TERN_X_BF16, tb.TERN_KV_I8, 2, Hkv, D, K, Hkv * D, V, Hkv * D, slots, pages, page, k, v, ks, vs)
    code, factor = quantise(K.reshape(2, Hkv, D), "i8")
    assert torch.equal(k[pages - 1, :, page - 1].cpu(), code[0])
    assert torch.equal(k[0, :, 3].cpu(), code[1])
    assert torch.equal(ks[pages - 1, :, page - 1].cpu(), factor[0])
    assert int((ks != 0).sum()) == 2 * Hkv
    Ko, Vo = torch.empty_like(K), torch.empty_like(V)
    tb.tern_kv_read(tb.TERN_X_BF16, tb.TERN_KV_I8, 2, Hkv, D, slots, pages, page, k, v, ks, vs, Ko, Hkv * D, Vo, Hkv * D)
    assert float((Ko.float() - K.float()).abs().max()) <= float(K.float().abs().max()) * (0.5 / 127 + 2.0 ** -8)


@pytest.mark.parametrize("kind", ["x16", "e4m3", "i8"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,t", [(3, 40, 8, 128, 128, "bf16"), (9, 6, 3, 96, 32, "f16"),
                                              (2, 64, 64, 64, 64, "bf16"), (4, 1, 1, 16, 0, "bf16")])
def test_rope_kv_write_is_the_two_calls(T, Hq, Hkv, D, rot, t, layout, kind):
    page, pages = 8, 4
    ld = (Hq + 2 * Hkv) * D
    qkv = heads(T + Hq, T, Hq + 2 * Hkv, D, t)
    q, k, v = qkv, qkv[:, Hq * D:], qkv[:, (Hq + Hkv) * D:]
    pos = positions(T, T).to(DEV)
    freq = torch.tensor(tb.tern_rope_freqs(max(rot, 2), 1e6)[0], dtype=torch.float32, device=DEV)
    slots = scatter_slots(T, T, pages, page).to(DEV)
    slots[0] = -1
    a, b = make_cache(pages, Hkv, page, D, kind, t), make_cache(pages, Hkv, page, D, kind, t)
    Qa, Qb = (torch.zeros((T, Hq * D), dtype=TYPES[t], device=DEV) for _ in range(2))
    Kr = torch.zeros((T, Hkv * D), dtype=TYPES[t], device=DEV)
    tb.tern_rope(X[t], LAYOUT[layout], T, D, rot, pos, freq, 1.1, Hq, q, ld, Qa, Hq * D, Hkv, k, ld, Kr, Hkv * D)
    tb.tern_kv_write(X[t], KV[kind], T, Hkv, D, Kr, Hkv * D, v, ld, slots, pages, page, *a)
    tb.tern_rope_kv_write(X[t], KV[kind], LAYOUT[layout], T, Hq, Hkv, D, rot, pos, freq, 1.1, q, ld, Qb, Hq * D, k, ld,
                          v, ld, slots, pages, page, *b)
    assert torch.equal(Qa.view(torch.int16), Qb.view(torch.int16))
    for x, y in zip(a, b):
        if x is not None:
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert not math.isnan(float(Qa.float().sum()))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,D,t", [(5, 16, 8, 80, "bf16"), (33, 3, 2, 48, "f16"), (3, 2, 1, 16, "bf16"),
                                         (4, 5, 3, 112, "bf16"), (3, 7, 2, 144, "f16"), (2, 3, 1, 240, "bf16")])
def test_rope_of_half_a_head(T, Hq, Hk, D, t, layout):
    """rot_dim an odd multiple of 8."""
    test_rope(T, Hq, Hk, D, D // 2, t, layout)


@pytest.mark.parametrize("kind", ["x16", "e4m3", "i8"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hkv,D,t", [(6, 8, 8, 80, "bf16"), (30, 6, 3, 48, "f16"), (3, 2, 1, 112, "bf16")])
def test_rope_kv_write_of_half_a_head(T, Hq, Hkv, D, t, layout, kind):
    test_rope_kv_write_is_the_two_calls(T, Hq, Hkv, D, D // 2, t, layout, kind)


def test_other_stream():
    """The calls run on the stream they are given."""
    T, H, D = 64, 8, 128
    Q = heads(1, T, H, D, "bf16")
    Qo, Qs = torch.empty_like(Q), torch.empty_like(Q)
    pos = positions(1, T).to(DEV)
    freq = torch.tensor(tb.tern_rope_freqs(D, 1e6)[0], dtype=torch.float32, device=DEV)
    args = (tb.TERN_X_BF16, tb.TERN_ROPE_HALF, T, D, D, pos, freq, 1.0, H, Q, H * D)
    tb.tern_rope(*args, Qo, H * D)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    tb.tern_rope(*args, Qs, H * D, stream=side)
    side.synchronize()
    assert torch.equal(Qo, Qs)


def test_random_reference_is_deterministic():
    assert torch.equal(randn(3, 4), randn(3, 4))
