"""Accumulated attention weights against 64-bit references.

Bounds.  A score is a sum of D exact products in fp32: off by at most D * 2^-23 *
scale * sum_d |q_d k_d| (S), and by 2^-21 of it for the scale's conversion to base
2, the row's power of two and the factor.  The logarithm's conversion adds
2^-23 |lse|, the sum's rounding and the exponential 2^-20.  With e the total, a
term is off by a relative e (1 + e); n terms add n * 2^-24 of their sum, terms
that fall below fp32's normal range 2^-126 each, and the joining with the old
weight 2^-23 of the result.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import TYPES, f64, heads, randn  # noqa: E402
from budget_util import KV, X16, Cache  # noqa: E402
from gpu_util import DEV  # noqa: E402
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402

pytestmark = pytest.mark.gpu


def scores(c, q, rows, b, h, G, scale):
    """[rows, room] scores of one sequence and head, and the sums of their magnitudes."""
    k = c.keys(b, h // G)
    x = f64(q[rows[0]:rows[1], h * c.D:(h + 1) * c.D])
    return x @ k.T * scale, np.abs(x) @ np.abs(k).T * scale


def reference(c, q, cu, lse, Hq, scale, known, decay, visible=None):
    """(weights, bound) of the whole plane."""
    G = Hq // c.Hkv
    want, bound = f64(c.weight).copy(), np.zeros(tuple(c.weight.shape))
    for b, n in enumerate(c.lens):
        nq = cu[b + 1] - cu[b]
        if nq <= 0 or n == 0:
            continue
        page, row = c.slots(b)
        ok = (page >= 0) & (page < c.pages) & (np.arange(len(page)) < n)
        for hk in range(c.Hkv):
            add, err = np.zeros(len(page)), np.zeros(len(page))
            for h in range(hk * G, (hk + 1) * G):
                s, S = scores(c, q, (cu[b], cu[b + 1]), b, h, G, scale)
                l = lse[cu[b]:cu[b + 1], h][:, None]
                j, i = np.arange(len(page)), np.arange(nq)[:, None]
                seen = (j <= i + n - nq) & ~np.isneginf(l)
                with np.errstate(invalid="ignore"):
                    p = np.where(seen, np.exp(np.where(seen, s - l, 0.0)), 0.0)
                    e = c.D * 2.0 ** -23 * S + 2.0 ** -21 * S + 2.0 ** -23 * np.abs(np.where(np.isneginf(l), 0, l)) + 2.0 ** -20
                add += p.sum(0)
                err += np.where(p > 0, p * e * (1 + e), 0).sum(0)
            old = f64(c.weight)[np.clip(page, 0, c.pages - 1), hk, row]
            new = np.where(np.arange(len(page)) < known[b], decay * old, 0.0) + add
            terms = nq * G
            want[page[ok], hk, row[ok]] = new[ok]
            bound[page[ok], hk, row[ok]] = (err + terms * 2.0 ** -24 * add + terms * 2.0 ** -126 + 2.0 ** -23 * np.abs(new))[ok]
    return want, bound


def run(c, q, ldq, cu, lse, Hq, scale, known, decay, x="bf16", single=False, stream=None):
    """The call, over a copy of the weights."""
    w = c.weight.clone()
    cu_dev = None if single else torch.tensor(cu, dtype=torch.int32, device=DEV)
    kn = None if known is None else torch.tensor(known, dtype=torch.int32, device=DEV)
    tb.tern_attn_weights(X16[x], KV[c.kv], len(c.lens), cu_dev, q.shape[0], Hq, c.Hkv, c.D, scale, q, ldq, lse, c.pages, c.page,
                         c.k, c.ks, c.dev_table, c.per, c.dev_lens, kn, decay, w, stream=stream)
    return w


def lse_of(c, q, cu, Hq, scale):
    """What attention reports for the rows."""
    out = np.full((cu[-1], Hq), -np.inf)
    for b, n in enumerate(c.lens):
        nq = cu[b + 1] - cu[b]
        for h in range(Hq):
            if nq <= 0 or n == 0:
                continue
            s, _ = scores(c, q, (cu[b], cu[b + 1]), b, h, Hq // c.Hkv, scale)
            seen = np.arange(s.shape[1]) <= np.arange(nq)[:, None] + n - nq
            m = np.where(seen, s, -np.inf).max(1)
            some = np.isfinite(m)
            m0 = np.where(some, m, 0)
            with np.errstate(divide="ignore"):
                out[cu[b]:cu[b + 1], h] = np.where(some, m0 + np.log(np.where(seen, np.exp(s - m0[:, None]), 0).sum(1)), -np.inf)
    return torch.tensor(out, dtype=torch.float32)


def check(got, want, bound, what=""):
    got = f64(got)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size}; first {np.argwhere(bad)[0]}: {got[bad][0]} {want[bad][0]} {bound[bad][0]}"


def case(seed, lens, rows, Hq, Hkv, D, page, kv, t, known=None, decay=1.0, pad=0, scale=None, single=False):
    c = Cache(seed, lens, Hkv, D, page, kv, t)
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    q = heads(seed + 20, cu[-1], Hq, D, t, pad=pad, spread=0.4)
    scale = D ** -0.5 if scale is None else scale
    scale = float(np.float32(scale))
    lse = lse_of(c, q, cu, Hq, scale)
    kn = [n - r for n, r in zip(lens, rows)] if known is None else known
    got = run(c, q, Hq * D + pad, cu, lse.to(DEV), Hq, scale, kn, decay, t, single)
    want, bound = reference(c, q, cu, f64(lse), Hq, scale, kn, decay)
    check(got, want, bound, f"{kv} {t}")
    return c, q, cu, lse, scale, got


@pytest.mark.parametrize("kv,t", [("x16", "bf16"), ("x16", "f16"), ("e4m3", "bf16"), ("i8", "f16"), ("i8", "bf16")])
@pytest.mark.parametrize("Hq,Hkv,D", [(10, 2, 128), (8, 8, 64), (3, 1, 80), (12, 1, 48), (17, 1, 16), (6, 3, 96), (40, 2, 112)])
def test_single_tokens(kv, t, Hq, Hkv, D):
    lens = [1, 700, 0, 15, 16, 17, 33, 64, 129, 257]
    rows = [min(1, n) for n in lens]
    case(Hq + D, lens, rows, Hq, Hkv, D, 16, kv, t, decay=0.9, pad=8)


@pytest.mark.parametrize("page", [1, 2, 4, 8, 32, 128, 1024])
@pytest.mark.parametrize("kv", ["x16", "i8"])
def test_pages(page, kv):
    case(page, [300, 1, 77, 513], [1, 1, 1, 1], 8, 2, 64, page, kv, "bf16", single=True)


@pytest.mark.parametrize("kv,t", [("x16", "bf16"), ("e4m3", "f16"), ("i8", "bf16"), ("x16", "f16")])
@pytest.mark.parametrize("lens,rows", [([40], [40]), ([300, 41], [7, 41]), ([130, 9, 0, 64], [130, 0, 0, 33]), ([513], [200]),
                                       ([5, 3], [9, 4]), ([128], [128]), ([1], [1]), ([257, 640], [64, 32])])
@pytest.mark.parametrize("Hq,Hkv,D", [(10, 2, 128), (2, 2, 64), (7, 1, 80), (20, 1, 48)])
def test_rows(kv, t, lens, rows, Hq, Hkv, D):
    """Windows, whole prompts, rows without tokens (more rows than tokens) and sequences without rows."""
    case(sum(lens) + D, lens, rows, Hq, Hkv, D, 16, kv, t, known=[max(0, n // 2) for n in lens], decay=0.5)


@pytest.mark.parametrize("page,kv,Hq,Hkv,D", [(4, "x16", 10, 2, 128), (1, "i8", 6, 2, 64), (8, "e4m3", 3, 1, 80),
                                              (16, "x16", 200, 1, 16), (32, "i8", 400, 2, 48)])
def test_many_rows_in_every_form(page, kv, Hq, Hkv, D):
    """Pages of fewer tokens than a copy takes, and more heads to a group than a column tile has."""
    case(page + Hq, [90, 140], [60, 9], Hq, Hkv, D, page, kv, "bf16", decay=0.5)


def test_one_prompt_among_idle_sequences():
    """The form is chosen by the average; a sequence of many rows is right in the form for few."""
    lens = [0] * 70 + [200] + [3] * 30
    case(44, lens, [0] * 70 + [150] + [0] * 30, 10, 2, 128, 16, "x16", "bf16")
    case(45, [130] + [5] * 90, [130] + [1] * 90, 8, 8, 64, 16, "i8", "f16")


def test_no_room_and_no_rows():
    """Tables of no pages, and calls whose sequences have nothing, change nothing."""
    c = Cache(3, [20, 30], 2, 64, 16, "x16", "bf16")
    q = heads(4, 4, 4, 64, "bf16")
    lse = torch.zeros((4, 4), device=DEV)
    before = c.weight.clone()
    for cu in ([0, 0, 0], [4, 4, 4]):
        assert torch.equal(run(c, q, 256, cu, lse, 4, 0.125, [0, 0], 1.0), before)
    w = c.weight.clone()
    tb.tern_attn_weights(0, 0, 2, torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV), 4, 4, 2, 64, 0.125, q, 256, lse, c.pages, 16,
                         c.k, None, None, 0, c.dev_lens, None, 1.0, w)
    assert torch.equal(w, before)


def test_many_sequences():
    """More than a warp has lanes, some idle."""
    lens = [(7 * b) % 90 for b in range(150)]
    case(3, lens, [1 if b % 5 else 0 for b in range(150)], 4, 2, 64, 16, "e4m3", "bf16")


def test_everything_known_by_default():
    c, q, cu, lse, scale, got = case(5, [50, 20], [1, 1], 4, 2, 64, 16, "x16", "bf16", known=[50, 20], decay=0.25)
    w = run(c, q, q.shape[1], cu, lse.to(DEV), 4, scale, None, 0.25)
    assert torch.equal(w, got)


def test_weights_of_a_row_add_to_one():
    """With attention's own logarithms every query head gives a weight of 1 in all."""
    B, Hq, Hkv, D, page = 5, 10, 2, 128, 16
    lens = [700, 1, 33, 500, 64]
    c = Cache(9, lens, Hkv, D, page, "i8", "bf16")
    q = heads(31, B, Hq, D, "bf16")
    o, lse = torch.empty_like(q), torch.empty((B, Hq), device=DEV)
    ws = torch.zeros(tb.tern_attn_decode_workspace_bytes(B, Hq, Hkv, D, c.per * page), dtype=torch.uint8, device=DEV)
    tb.tern_attn_decode(0, KV["i8"], B, Hq, Hkv, D, D ** -0.5, q, Hq * D, c.pages, page, c.k, c.v, c.ks, c.vs, c.dev_table, c.per,
                        c.dev_lens, o, Hq * D, lse, ws)
    c.weight.zero_()
    w = f64(run(c, q, Hq * D, None, lse, Hq, D ** -0.5, [0] * B, 1.0, single=True))
    for b, n in enumerate(lens):
        p, r = c.slots(b)
        total = w[p[:n], :, r[:n]].sum(0)
        # a softmax off by its scores' error on both sides: 2 * D * 2^-23 * S, S below 100 here
        assert np.abs(total - Hq / Hkv).max() <= Hq / Hkv * (2 * D * 2.0 ** -23 * 100 + 2.0 ** -18)


@pytest.mark.parametrize("kv", ["x16", "e4m3"])
def test_what_is_not_there_is_not_read(kv):
    """NaN in cells behind the last token, in unknown weights and in hidden pages; hidden tokens keep their weight."""
    c = Cache(2, [100, 40], 2, 64, 16, kv, "bf16")
    c.table[0, 2], c.table[1, 1] = -1, c.pages + 5
    c.dev_table = c.table.to(DEV)
    for b, n in enumerate(c.lens):
        p, r = c.slots(b)
        for j in range(n, len(p)):
            if 0 <= p[j] < c.pages:
                if kv == "x16":
                    c.k[p[j], :, r[j]] = float("nan")
                else:
                    c.ks[p[j], :, r[j]] = float("nan")
        if 0 <= p[n - 1] < c.pages:
            c.weight[p[n - 1], :, r[n - 1]] = float("nan")
    q = heads(4, 2, 6, 64, "bf16")
    lse = torch.tensor([[1.0, 2.0, 3.0, 1.0, 2.0, 3.0]] * 2)
    kept = c.weight.clone()
    c.weight = torch.nan_to_num(c.weight)
    want, bound = reference(c, q, [0, 1, 2], f64(lse), 6, 0.125, [99, 39], 1.0)
    c.weight = kept
    got = run(c, q, 384, [0, 1, 2], lse.to(DEV), 6, 0.125, [99, 39], 1.0)
    check(got, want, bound)


def test_what_is_not_finite_stays_with_its_token():
    c = Cache(6, [70], 1, 64, 16, "x16", "bf16")
    p, r = c.slots(0)
    c.k[p[20], 0, r[20], 5] = float("nan")
    q = heads(7, 1, 3, 64, "bf16")
    w = run(c, q, 192, [0, 1], torch.zeros((1, 3), device=DEV), 3, 0.125, [69], 1.0)
    bad = torch.isnan(w).nonzero().tolist()
    assert bad == [[int(p[20]), 0, int(r[20])]]
    # a row with an infinite key: its weight where the score is -infinity is none
    c = Cache(6, [70], 1, 64, 16, "x16", "bf16")
    c.k[p[20], 0, r[20], 5] = float("inf")
    q[0, 5], q[0, 64 + 5], q[0, 128 + 5] = -1.0, -2.0, -0.5
    w = run(c, q, 192, [0, 1], torch.zeros((1, 3), device=DEV), 3, 0.125, [0], 1.0)
    assert torch.isfinite(w).all() and w[p[20], 0, r[20]] == 0.0


@pytest.mark.parametrize("kv", ["x16", "i8"])
def test_sizes_of_values(kv):
    """Large scores with logarithms to match, tiny queries, a scale of zero."""
    for size, scale in ((60.0, 0.125), (2.0 ** -120, 0.125), (1.0, 0.0)):
        c = Cache(8, [90], 2, 64, 16, kv, "bf16")
        q = (randn(3, 2, 4 * 64) * size).to(torch.bfloat16).to(DEV)
        lse = lse_of(c, q, [0, 2], 4, scale)
        got = run(c, q, 256, [0, 2], lse.to(DEV), 4, scale, [88], 1.0)
        want, bound = reference(c, q, [0, 2], f64(lse), 4, scale, [88], 1.0)
        check(got, want, bound, f"{size}")


def test_offsets_outside_are_read_as_the_nearest_end():
    c = Cache(12, [60, 30, 20], 2, 64, 16, "x16", "bf16")
    q = heads(13, 5, 4, 64, "bf16")
    lse = lse_of(c, q, [0, 2, 4, 5], 4, 0.125)
    want = run(c, q, 256, [0, 2, 4, 5], lse.to(DEV), 4, 0.125, [0, 0, 0], 1.0)
    got = run(c, q, 256, [-7, 2, 4, 900], lse.to(DEV), 4, 0.125, [0, 0, 0], 1.0)
    assert torch.equal(got, want)
    before = c.weight.clone()
    got = run(c, q, 256, [5, 3, 3, 0], lse.to(DEV), 4, 0.125, [0, 0, 0], 1.0)
    assert torch.equal(got, before)


def test_lengths_past_the_table_and_far_cells():
    """A length past the table's room; keys more than 2^32 bytes into the cache."""
    c = Cache(14, [64, 30], 2, 64, 16, "x16", "bf16")
    q = heads(15, 2, 4, 64, "bf16")
    lse = lse_of(c, q, [0, 1, 2], 4, 0.125)
    want = run(c, q, 256, [0, 1, 2], lse.to(DEV), 4, 0.125, [63, 29], 1.0)
    c.dev_lens = torch.tensor([100000, 30], dtype=torch.int32, device=DEV)
    assert torch.equal(run(c, q, 256, [0, 1, 2], lse.to(DEV), 4, 0.125, [63, 29], 1.0), want)

    pages, page, D = 280000, 64, 128     # 4.6 GB of keys
    k = torch.zeros((pages, 1, page, D), dtype=torch.bfloat16, device=DEV)
    far = Cache(16, [2 * page], 1, D, page, "x16", "bf16")
    q = heads(17, 1, 4, D, "bf16")
    lse = lse_of(far, q, [0, 1], 4, D ** -0.5)
    want = run(far, q, 512, [0, 1], lse.to(DEV), 4, D ** -0.5, [0], 1.0)
    k[-2:] = far.k[far.table[0].long()]
    w = torch.zeros((pages, 1, page), device=DEV)
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device=DEV)
    tb.tern_attn_weights(0, 0, 1, None, 1, 4, 1, D, D ** -0.5, q, 512, lse.to(DEV), pages, page, k, None, table, 2, far.dev_lens,
                         torch.zeros(1, dtype=torch.int32, device=DEV), 1.0, w)
    assert torch.equal(w[-2:], want[far.table[0].long()])
    assert int((w != 0).sum()) == 2 * page


def test_repeats_streams_and_graphs():
    """The same bits every time; on a stream of its own; captured and replayed on new lengths."""
    c, q, cu, lse, scale, got = case(18, [1000, 300, 77], [40, 1, 9], 10, 2, 128, 16, "e4m3", "bf16")
    lse = lse.to(DEV)
    kn = [960, 299, 68]
    for _ in range(5):
        assert torch.equal(run(c, q, 1280, cu, lse, 10, scale, kn, 1.0), got)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w = run(c, q, 1280, cu, lse, 10, scale, kn, 1.0)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(w, got)
    w = c.weight.clone()
    cu_dev, kn_dev = torch.tensor(cu, dtype=torch.int32, device=DEV), torch.tensor(kn, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tb.tern_attn_weights(0, KV["e4m3"], 3, cu_dev, q.shape[0], 10, 2, 128, scale, q, 1280, lse, c.pages, 16, c.k, c.ks,
                             c.dev_table, c.per, c.dev_lens, kn_dev, 1.0, w)
    c.lens = [500, 300, 30]
    c.dev_lens.copy_(torch.tensor(c.lens))
    w.copy_(c.weight)
    graph.replay()
    want, bound = reference(c, q, cu, f64(lse), 10, scale, kn, 1.0)
    check(w, want, bound, "replayed")


@pytest.mark.parametrize("kv", ["e4m3", "i8"])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_weights_of_a_prompt_over_codes_add_to_its_rows(kv, t):
    """tern_attn_prompt's logarithms are of the keys that tern_kv_read rounded to 16 bits, the weights of the keys before
    that: a row's scores differ by u S, u the type's half step, beside both calls' own errors."""
    lens, rows, Hq, Hkv, D, page = [300, 130], [300, 40], 10, 2, 128, 16
    c = Cache(17, lens, Hkv, D, page, kv, t)
    q = heads(33, sum(rows), Hq, D, t, spread=0.2)
    slots = torch.cat([torch.from_numpy(p[:n].astype(np.int64) * page + r[:n]) for n, (p, r) in
                       ((n, c.slots(b)) for b, n in enumerate(lens))]).to(DEV)
    k, v = (torch.empty((sum(lens), Hkv * D), dtype=TYPES[t], device=DEV) for _ in range(2))
    tb.tern_kv_read(X16[t], KV[kv], sum(lens), Hkv, D, slots, c.pages, page, c.k, c.v, c.ks, c.vs, k, Hkv * D, v, Hkv * D)
    cu_q, cu_k = (torch.tensor([0, *np.cumsum(x)], dtype=torch.int32, device=DEV) for x in (rows, lens))
    o, lse = torch.empty_like(q), torch.empty((sum(rows), Hq), device=DEV)
    ws = torch.zeros(tb.tern_attn_prompt_workspace_bytes(2, sum(rows), sum(lens), Hq, Hkv, D), dtype=torch.uint8, device=DEV)
    scale = float(np.float32(D ** -0.5))
    tb.tern_attn_prompt(X16[t], 2, cu_q, cu_k, sum(rows), sum(lens), Hq, Hkv, D, True, scale, q, Hq * D, k, Hkv * D, v, Hkv * D, o,
                        Hq * D, lse, ws)
    cu = cu_q.tolist()
    w = f64(run(c, q, Hq * D, cu, lse, Hq, scale, [0, 0], 1.0, t))
    for b, n in enumerate(lens):
        p, r = c.slots(b)
        for g in range(Hkv):
            S = max(scores(c, q, (cu[b], cu[b + 1]), b, h, Hq // Hkv, scale)[1].max() for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv))
            e = (2.0 ** -8 if t == "bf16" else 2.0 ** -11) * S + 2 * (D * 2.0 ** -23 * S + 2.0 ** -20) + 2.0 ** -20 * np.abs(f64(lse)).max()
            want = rows[b] * Hq // Hkv
            assert abs(w[p[:n], g, r[:n]].sum() - want) <= want * np.expm1(e)
