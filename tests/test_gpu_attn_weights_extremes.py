"""Accumulated attention weights of scores, queries, factors and logarithms at the ends of their
types' range, in each of the three forms.

Where every score is one product that fp32 holds exactly, the only roundings before the
exponential are that of score - logarithm, relative 2^-24 (and for codes the product of factor
and scale, 2^-24 of the score, where the scale is not a power of two), and that of its
conversion to base 2, two of 2^-24: with x the difference, a weight is off by a relative
3 * 2^-24 |x| and by 2^-20 for the exponential and the sums.  A weight beyond fp32 is infinite.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import TYPES, f64, heads  # noqa: E402
from budget_util import Cache  # noqa: E402
from gpu_util import DEV  # noqa: E402
from test_gpu_attn_weights import check, lse_of, reference, run  # noqa: E402

pytestmark = pytest.mark.gpu

# page, rows of each sequence: keys that come by TMA; small pages; many rows
FORMS = [(16, [1, 1]), (4, [1, 1]), (16, [9, 30])]
LENS = [130, 41]
HQ, HKV = 4, 2


def one_product(q, k, t, kv, page, rows, D, scale):
    """A cache whose scores are all scale * q * k, one product each: (cache, queries, offsets, score)."""
    c = Cache(3, LENS, HKV, D, page, kv, t)
    c.k.zero_()
    key = float(torch.tensor(k, dtype=TYPES[t]))
    if kv == "x16":
        c.k[..., 0] = key
    else:
        c.k[..., 0] = (0x7E if kv == "e4m3" else 127) if k > 0 else (0xFE if kv == "e4m3" else 129)
        top = 448.0 if kv == "e4m3" else 127.0
        c.ks.fill_(abs(key) / top)
        key = float(c.ks.reshape(-1)[0]) * top * (1 if k > 0 else -1)
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    Q = torch.zeros((cu[-1], HQ * D), dtype=TYPES[t], device=DEV)
    Q[:, ::D] = q
    return c, Q, cu, float(Q[0, 0]) * key * float(np.float32(scale))


@pytest.mark.parametrize("page,rows", FORMS)
@pytest.mark.parametrize("q,k,t,scale", [
    (3001.0, 3001.0, "f16", 1.0),           # 9e6: the score's unit is 1
    (60000.0, -60000.0, "f16", 1.0),        # 3.6e9: the unit is 256
    (7e5, 7e5, "bf16", 0.125), (250.0, 250.0, "bf16", 0.7),
    (1.5e19, -1.5e19, "bf16", 1.0), (1.5e19, 1.5e19, "bf16", 1.0),
    (2.0 ** -60, 2.0 ** -60, "bf16", 3e38), (2.0 ** -60, -2.0 ** -60, "bf16", 3e38), (0.0, 1.0, "bf16", 3e38)])
@pytest.mark.parametrize("kv,D", [("x16", 64), ("x16", 128), ("e4m3", 64), ("i8", 128)])
def test_one_product(page, rows, q, k, t, scale, kv, D):
    """Equal scores of any size, with the logarithms of their sums."""
    c, Q, cu, score = one_product(q, k, t, kv, page, rows, D, scale)
    lse = np.zeros((cu[-1], HQ))
    for b, (n, r) in enumerate(zip(LENS, rows)):
        lse[cu[b]:cu[b + 1]] = score + np.log(np.arange(r) + 1 + n - r)[:, None]
    lse = torch.tensor(lse, dtype=torch.float32)
    got = f64(run(c, Q, HQ * D, cu, lse.to(DEV), HQ, scale, [0, 0], 1.0, t))
    G = HQ // HKV
    for b, (n, r) in enumerate(zip(LENS, rows)):
        page_, row_ = c.slots(b)
        x = score - f64(lse[cu[b]:cu[b + 1], 0])
        seen = np.arange(n) <= np.arange(r)[:, None] + n - r
        with np.errstate(over="ignore", invalid="ignore"):
            term = np.exp(x)
            term = np.where(term > 3.5e38, np.inf, np.where(term < 2.0 ** -126, 0.0, term))[:, None]
            err = term * (3 * 2.0 ** -24 * np.abs(x)[:, None] + 2.0 ** -20)
            if kv != "x16":
                err = err + term * 2.0 ** -24 * abs(score)
            want, bound = (G * np.where(seen, y, 0.0).sum(0) for y in (term, err))
        mine = got[page_[:n], :, row_[:n]]
        with np.errstate(invalid="ignore"):
            ok = (np.abs(mine - want[:, None]) <= bound[:, None] + 2.0 ** -120) | (mine == want[:, None])
        assert ok.all(), (b, mine[~ok][0], np.broadcast_to(want[:, None], mine.shape)[~ok][0])


@pytest.mark.parametrize("page,rows", FORMS)
@pytest.mark.parametrize("kv", ["e4m3", "i8"])
@pytest.mark.parametrize("power", [-98, -102, -106, -108, -112, -116])
def test_tiny_queries_against_large_keys(page, rows, kv, power):
    """Queries times 2^power, factors times 2^5 / 2^power: scores of some tens."""
    D = 128
    c = Cache(13, LENS, HKV, D, page, kv, "bf16")
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    Q = (heads(14, cu[-1], HQ, D, "bf16").double() * 2.0 ** power).to(torch.bfloat16)
    c.ks = (c.ks.double() * 2.0 ** (5 - power)).float()
    assert torch.isfinite(c.ks).all()
    scale = float(np.float32(D ** -0.5))
    lse = lse_of(c, Q, cu, HQ, scale)
    want, bound = reference(c, Q, cu, f64(lse), HQ, scale, [0, 0], 1.0)
    check(run(c, Q, HQ * D, cu, lse.to(DEV), HQ, scale, [0, 0], 1.0), want, bound, f"2^{power}")


@pytest.mark.parametrize("page,rows", FORMS)
@pytest.mark.parametrize("kv,t", [("x16", "bf16"), ("x16", "f16"), ("e4m3", "bf16"), ("i8", "f16")])
def test_rows_that_saw_nothing_add_nothing_whatever_they_hold(page, rows, kv, t):
    """A row whose logarithm is -infinity, of NaN and infinities, between rows that have weights."""
    D = 64
    c = Cache(5, LENS, HKV, D, page, kv, t)
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    Q = heads(6, cu[-1], HQ, D, t)
    lse = lse_of(c, Q, cu, HQ, 0.125)
    for i, x in ((0, float("nan")), (cu[-1] - 1, float("inf"))):
        Q[i, :D] = x                    # one head of two that share keys
        lse[i, 0] = float("-inf")
    finite = torch.nan_to_num(Q, nan=0.0, posinf=0.0)
    want, bound = reference(c, finite, cu, f64(lse), HQ, 0.125, [0, 0], 1.0)
    check(run(c, Q, HQ * D, cu, lse.to(DEV), HQ, 0.125, [0, 0], 1.0, t), want, bound)


@pytest.mark.parametrize("page,rows", FORMS)
@pytest.mark.parametrize("kv", ["e4m3", "i8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [100, 104, 108, 111, 113, 115, 117, 118, -100, -108, -112, -116, -120])
def test_queries_and_factors_that_make_up_for_one_another(page, rows, kv, D, power):
    """Queries times 2^power, factors divided by it: the scores stay of ordinary size while their
    products with the codes would leave fp32's range, or fall below it."""
    c = Cache(7, LENS, HKV, D, page, kv, "bf16")
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    Q = (heads(8, cu[-1], HQ, D, "bf16").double() * 2.0 ** power).to(torch.bfloat16)
    c.ks = (c.ks.double() * 2.0 ** -power).float()
    assert torch.isfinite(c.ks).all() and torch.isfinite(Q.float()).all()
    scale = float(np.float32(D ** -0.5))
    lse = lse_of(c, Q, cu, HQ, scale)
    want, bound = reference(c, Q, cu, f64(lse), HQ, scale, [0, 0], 1.0)
    check(run(c, Q, HQ * D, cu, lse.to(DEV), HQ, scale, [0, 0], 1.0), want, bound, f"2^{power}")


@pytest.mark.parametrize("kv", ["e4m3", "i8"])
@pytest.mark.parametrize("page,rows", FORMS)
def test_some_rows_and_keys_far_from_the_others(page, rows, kv):
    """Rows of ordinary size and rows of 2^115, against keys whose factors undo that (to rows of ordinary
    size they are next to nothing) and keys of ordinary factors that are zero."""
    D = 128
    c = Cache(9, LENS, HKV, D, page, kv, "bf16")
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    Q = heads(10, cu[-1], HQ, D, "bf16")
    far = (torch.arange(cu[-1]) % 3 == 1).to(DEV)
    Q = torch.where(far[:, None], (Q.double() * 2.0 ** 115).to(torch.bfloat16), Q)
    c.ks[:, :, ::2] = (c.ks[:, :, ::2].double() * 2.0 ** -115).float()
    c.k[:, :, 1::2] = 0
    scale = float(np.float32(D ** -0.5))
    lse = lse_of(c, Q, cu, HQ, scale)
    want, bound = reference(c, Q, cu, f64(lse), HQ, scale, [0, 0], 1.0)
    check(run(c, Q, HQ * D, cu, lse.to(DEV), HQ, scale, [0, 0], 1.0), want, bound)


@pytest.mark.parametrize("kv", ["e4m3", "i8"])
@pytest.mark.parametrize("page,rows", FORMS)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_a_factor_that_is_not_a_number_stays_with_its_token(page, rows, kv, t):
    """NaN and zero factors: the token's weight is NaN, or that of a score of zero."""
    D = 64
    c = Cache(11, LENS, HKV, D, page, kv, t)
    p, r = c.slots(0)
    c.ks[p[5], 0, r[5]], c.ks[p[20], 1, r[20]] = 0.0, float("nan")
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    Q = heads(12, cu[-1], HQ, D, t)
    lse = torch.full((cu[-1], HQ), 3.0)
    got = run(c, Q, HQ * D, cu, lse.to(DEV), HQ, 0.125, [0, 0], 1.0, t)
    assert torch.isnan(got).nonzero().tolist() == [[int(p[20]), 1, int(r[20])]]
    c.ks[p[20], 1, r[20]] = 1.0
    want, bound = reference(c, Q, cu, f64(lse), HQ, 0.125, [0, 0], 1.0)
    skip = (int(p[20]), 1, int(r[20]))
    got[skip], want[skip] = 0.0, 0.0
    check(got, want, bound)
