"""Attention of scores, queries, keys and values at the ends of their types' range.

Where scores are large, an error of 2^-24 of a score is many units of the
exponent and the softmax of unequal scores is not determined by the inputs'
bits; these tests use equal scores (the weights are then equal, whatever
their size) or scores that differ by more than any rounding (the largest takes
all).  Equal weights: the output is the mean of n values, each weight is the
same 16-bit number w and the sum takes n times w unrounded, so it is within
u |o| + (u + n 2^-23) max |v| of the mean (u covers the rounding of w)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import TYPES, UNIT, assert_close, f64, heads  # noqa: E402
from gpu_util import DEV  # noqa: E402
from test_gpu_attention import make_cache, run_decode, run_prompt  # noqa: E402

pytestmark = pytest.mark.gpu

# Rows and keys: one tile per CTA; two tiles; keys split over CTAs.
SIZES = [([40], [40], 2, 1, 128), ([900, 70], [900, 900], 16, 8, 64), ([16], [2100], 4, 1, 128)]


def mean_rows(V, n, m, causal):
    """[n, D] means of the values that rows 0 .. n-1 see of m keys."""
    total = np.concatenate([np.zeros((1, V.shape[1])), np.cumsum(V, 0)])
    seen = np.clip(np.arange(n) + 1 + m - n, 0, m) if causal else np.full(n, m)
    return total[seen] / np.maximum(seen, 1)[:, None], seen


def check_means(O, L, V, nq, nk, Hq, Hkv, D, t, causal, score):
    o, l, v = f64(O), f64(L), f64(V)
    a = c = 0
    for n, m in zip(nq, nk):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            vv = v[c:c + m, g * D:(g + 1) * D]
            want, seen = mean_rows(vv, n, m, causal)
            bound = UNIT[t] * np.abs(want) + (UNIT[t] + m * 2.0 ** -23) * np.abs(vv).max()
            assert_close(o[a:a + n, h * D:(h + 1) * D], want, bound, f"head {h}")
            lse = score + np.log(seen)
            assert_close(l[a:a + n, h], lse, 1e-6 * np.abs(lse) + 1e-5, f"lse of head {h}")
        a, c = a + n, c + m


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D", SIZES)
@pytest.mark.parametrize("q,k,t", [
    (1.5e19, 1.5e19, "bf16"),
    (3001.0, 3001.0, "f16"),        # 9e6: the score's unit is 1
    (60000.0, -60000.0, "f16"),     # 3.6e9: the unit is 256 and more
    (7e5, 7e5, "bf16"),
])
def test_prompt_of_equal_scores(q, k, t, nq, nk, Hq, Hkv, D, causal):
    prompt_of_equal_scores(q, k, t, nq, nk, Hq, Hkv, D, causal)


def prompt_of_equal_scores(q, k, t, nq, nk, Hq, Hkv, D, causal):
    Q, K = (torch.zeros((sum(n), H * D), dtype=TYPES[t], device=DEV) for n, H in ((nq, Hq), (nk, Hkv)))
    Q[:, ::D] = q
    K[:, ::D] = k
    V = heads(1, sum(nk), Hkv, D, t)
    O, L = run_prompt(Q, K, V, nq, nk, Hq, Hkv, D, t, causal, 1.0)
    score = float(Q[0, 0].double() * K[0, 0].double())
    check_means(O, L, V, nq, nk, Hq, Hkv, D, t, causal, score)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D", SIZES)
def test_prompt_of_far_scores(nq, nk, Hq, Hkv, D, t):
    """One key is ahead of all others by far: every row takes its value."""
    Q = torch.full((sum(nq), Hq * D), 2000.0, dtype=TYPES[t], device=DEV)
    K = torch.full((sum(nk), Hkv * D), 2000.0, dtype=TYPES[t], device=DEV)
    V = heads(2, sum(nk), Hkv, D, t)
    c = a = 0
    for m in nk:
        K[c + m // 3] = 3001.0
        c += m
    O, L = run_prompt(Q, K, V, nq, nk, Hq, Hkv, D, t, False, 1.0)
    score = float((Q[0, :D].double() * K[nk[0] // 3, :D].double()).sum())
    assert torch.all((L.double() - score).abs() <= 1e-5 * score)
    c = 0
    for n, m in zip(nq, nk):
        want = V[c + m // 3].reshape(Hkv, 1, D).expand(Hkv, Hq // Hkv, D).reshape(Hq * D)
        # the weight 2^0 .. 2^8 of the one key cancels up to two roundings
        assert torch.allclose(O[a:a + n, :Hq * D].float(), want.float().expand(n, -1), rtol=2 * UNIT[t], atol=0)
        a, c = a + n, c + m


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D", SIZES)
def test_prompt_of_lowest_scores(nq, nk, Hq, Hkv, D, causal):
    """-2.3e38, in base 2 -3.3e38: the far end of what is finite."""
    prompt_of_equal_scores(1.5e19, -1.5e19, "bf16", nq, nk, Hq, Hkv, D, causal)


DECODES = [([40, 700], 4, 2, 128), ([9000], 2, 1, 64), ([130], 12, 1, 128)]


def decode_of_equal_scores(q, k, t, lens, Hq, Hkv, D, kind):
    B = len(lens)
    Q = torch.zeros((B, Hq * D), dtype=TYPES[t], device=DEV)
    Q[:, ::D] = q
    pages, cache, table, plain = make_cache(lens, Hkv, 16, D, kind, t, 6)
    cache[0].zero_()
    key = float(torch.tensor(k, dtype=TYPES[t]))
    if kind == "x16":
        cache[0][..., 0] = key
    else:
        # the largest code and its factor, as a write of such keys makes them
        cache[0][..., 0] = (0x7E if kind == "e4m3" else 127) if k > 0 else (0xFE if kind == "e4m3" else 129)
        top = 448.0 if kind == "e4m3" else 127.0
        cache[2].fill_(abs(key) / top)
        key = float(cache[2].reshape(-1)[0]) * top * (1 if k > 0 else -1)
    O, L = run_decode(Q, lens, Hq, Hkv, D, 16, kind, t, 1.0, pages, cache, table)
    score = float(Q[0, 0]) * key
    o, l = f64(O), f64(L)
    u = UNIT[t if kind == "x16" else "f16"]
    for b, n in enumerate(lens):
        for h in range(Hq):
            v = plain[1][b][h // (Hq // Hkv)]
            want = v.mean(0)
            assert_close(o[b, h * D:(h + 1) * D], want, UNIT[t] * np.abs(want) + (u + n * 2.0 ** -23) * np.abs(v).max(), f"head {h}")
            assert_close(l[b, h], score + np.log(n), 1e-6 * abs(score) + 1e-5, f"lse of head {h}")


@pytest.mark.parametrize("lens,Hq,Hkv,D", DECODES)
@pytest.mark.parametrize("q,k,t", [(1.5e19, -1.5e19, "bf16"), (60000.0, -60000.0, "f16"), (7e5, 7e5, "bf16")])
def test_decode_of_equal_scores(q, k, t, lens, Hq, Hkv, D):
    decode_of_equal_scores(q, k, t, lens, Hq, Hkv, D, "x16")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D", SIZES)
def test_prompt_of_scale_zero(nq, nk, Hq, Hkv, D, causal):
    """Scale zero weighs all keys alike, however large the products are."""
    Q, K, V = (heads(s, n, H, D, "bf16") for s, n, H in ((3, sum(nq), Hq), (4, sum(nk), Hkv), (5, sum(nk), Hkv)))
    Q *= 2.0 ** 60
    K *= 2.0 ** 50
    O, L = run_prompt(Q, K, V, nq, nk, Hq, Hkv, D, "bf16", causal, 0.0)
    check_means(O, L, V, nq, nk, Hq, Hkv, D, "bf16", causal, 0.0)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("lens,Hq,Hkv,D", DECODES)
@pytest.mark.parametrize("q,k,t", [(100.0, 100.0, "bf16"), (3001.0, 3001.0, "f16"), (60000.0, -60000.0, "f16"),
                                   (7e5, 7e5, "bf16"), (1.5e19, -1.5e19, "bf16"), (1.5e19, 1.5e19, "bf16")])
def test_decode_of_equal_scores_over_codes(q, k, t, lens, Hq, Hkv, D, kind):
    """Value factors of unequal size under large scores."""
    decode_of_equal_scores(q, k, t, lens, Hq, Hkv, D, kind)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("size", [2.0 ** -110, 2.0 ** -124])
def test_decode_of_tiny_queries(size, kind):
    """Queries at the small end of bf16 against keys at the large end: the scores are
    of ordinary size (powers of two move between the two without a rounding)."""
    lens, Hq, Hkv, D, t = [300, 17], 4, 2, 64, "bf16"
    Q = heads(7, 2, Hq, D, t)
    pages, cache, table, plain = make_cache(lens, Hkv, 16, D, kind, t, 8)
    small = (Q.double() * size).to(TYPES[t])
    keep = small.double() / size == Q.double()     # what is below bf16's range drops out in both
    cache[2] *= 1.0 / size
    O1, L1 = run_decode(torch.where(keep, Q, torch.zeros_like(Q)), lens, Hq, Hkv, D, 16, kind, t, 0.125, pages,
                        [cache[0], cache[1], cache[2] * size, cache[3]], table)
    O2, L2 = run_decode(torch.where(keep, small, torch.zeros_like(Q)), lens, Hq, Hkv, D, 16, kind, t, 0.125, pages, cache, table)
    # scores of the two calls differ by fp32 roundings at most: their bound in attn_util.py, twice
    assert torch.allclose(L1, L2, rtol=2.0 ** -16, atol=2.0 ** -14)
    assert torch.allclose(O1[:, :Hq * D].float(), O2[:, :Hq * D].float(), rtol=2.0 ** -6, atol=2.0 ** -8)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -121])
def test_decode_of_tiny_values(size, kind):
    """Values at the small end of bf16: the output is the value of the same call scaled by a power of two."""
    lens, Hq, Hkv, D, t = [200, 1], 4, 2, 64, "bf16"
    Q = heads(9, 2, Hq, D, t)
    pages, cache, table, plain = make_cache(lens, Hkv, 16, D, kind, t, 10)
    O1, L1 = run_decode(Q, lens, Hq, Hkv, D, 16, kind, t, 0.125, pages, cache, table)
    cache[3] *= size
    O2, L2 = run_decode(Q, lens, Hq, Hkv, D, 16, kind, t, 0.125, pages, cache, table)
    assert torch.equal(L1, L2)
    o1, o2 = O1[:, :Hq * D].double(), O2[:, :Hq * D].double() / size
    # beside the roundings of both calls, half of bf16's smallest number
    assert torch.all((o1 - o2).abs() <= 2 * UNIT[t] * o1.abs() + 2.0 ** -133 / size)


def one_sided_means(V, n, m, causal, ahead):
    """Means over the visible keys from `ahead` on, or over all that are visible where none is."""
    out = np.zeros((n, V.shape[1]))
    for i in range(n):
        seen = min(m, max(0, i + 1 + m - n)) if causal else m
        if seen > 0:
            out[i] = V[ahead:seen].mean(0) if seen > ahead else V[:seen].mean(0)
    return out


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ahead", [20, 128, 300, 700])
def test_prompt_of_scores_across_the_whole_range(ahead, causal):
    """Keys with scores of -2.3e38 before keys with 2.3e38: their distance is beyond fp32."""
    for n, m, Hq, Hkv, D in ((900, 900, 16, 8, 64), (40, 1000, 2, 1, 128), (16, 2100, 4, 1, 128)):
        Q, K = (torch.zeros((r, H * D), dtype=torch.bfloat16, device=DEV) for r, H in ((n, Hq), (m, Hkv)))
        Q[:, ::D] = 1.5e19
        K[:ahead, ::D] = -1.5e19
        K[ahead:, ::D] = 1.5e19
        V = heads(11, m, Hkv, D, "bf16")
        O, L = run_prompt(Q, K, V, [n], [m], Hq, Hkv, D, "bf16", causal, 1.0)
        o, v = f64(O), f64(V)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            vv = v[:, g * D:(g + 1) * D]
            want = one_sided_means(vv, n, m, causal, ahead)
            bound = UNIT["bf16"] * np.abs(want) + (UNIT["bf16"] + m * 2.0 ** -23) * np.abs(vv).max()
            assert_close(o[:, h * D:(h + 1) * D], want, bound, f"head {h}")


@pytest.mark.parametrize("ahead", [5, 16, 300])
def test_decode_of_scores_across_the_whole_range(ahead):
    Hq, Hkv, D, n = 4, 2, 64, 700
    Q = torch.zeros((1, Hq * D), dtype=torch.bfloat16, device=DEV)
    Q[:, ::D] = 1.5e19
    pages, cache, table, plain = make_cache([n], Hkv, 16, D, "x16", "bf16", 12)
    cache[0].zero_()
    for j in range(n):
        cache[0][int(table[0, j // 16]), :, j % 16, 0] = -1.5e19 if j < ahead else 1.5e19
    O, L = run_decode(Q, [n], Hq, Hkv, D, 16, "x16", "bf16", 1.0, pages, cache, table)
    o = f64(O)
    for h in range(Hq):
        v = plain[1][0][h // (Hq // Hkv)]
        want = v[ahead:].mean(0)
        assert_close(o[0, h * D:(h + 1) * D], want, UNIT["bf16"] * np.abs(want) + (UNIT["bf16"] + n * 2.0 ** -23) * np.abs(v).max(), f"head {h}")
