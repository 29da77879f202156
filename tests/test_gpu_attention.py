"""Attention over packed prompts and over the paged cache against a 64-bit
reference (bounds: attn_util.py)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import TYPES, assert_close, attend, bounds, code_values, f64, heads, quantise  # noqa: E402
from gpu_util import DEV  # noqa: E402
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402

pytestmark = pytest.mark.gpu

X = {"bf16": tb.TERN_X_BF16, "f16": tb.TERN_X_F16}
KV = {"x16": tb.TERN_KV_X16, "e4m3": tb.TERN_KV_E4M3, "i8": tb.TERN_KV_I8}


def cumulative(lens, gap=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]) + gap, dtype=torch.int32)


def workspace(nbytes):
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=DEV)


def run_prompt(Q, K, V, nq, nk, Hq, Hkv, D, t, causal, scale, gap=0, lse=True, O=None, ws=None, stream=None):
    Tq, Tkv = Q.shape[0], K.shape[0]
    cu_q, cu_k = cumulative(nq, gap).to(DEV), cumulative(nk, gap).to(DEV)
    O = torch.full((Tq, Hq * D + 8), 7.0, dtype=TYPES[t], device=DEV) if O is None else O
    L = torch.full((Tq, Hq), 7.0, device=DEV) if lse else None
    ws = workspace(tb.tern_attn_prompt_workspace_bytes(len(nq), Tq, Tkv, Hq, Hkv, D)) if ws is None else ws
    tb.tern_attn_prompt(X[t], len(nq), cu_q, cu_k, Tq, Tkv, Hq, Hkv, D, causal, scale, Q, Q.stride(0), K, K.stride(0),
                        V, V.stride(0), O, O.stride(0), L, ws, stream=stream)
    if stream is not None:
        stream.synchronize()
    assert tb.tern_workspace_error(ws) == 0
    return O, L


def check_prompt(Q, K, V, O, L, nq, nk, Hq, Hkv, D, t, causal, scale, gap=0, only=None):
    """Every row of every sequence against the reference; rows of no sequence untouched."""
    q, k, v, o = f64(Q), f64(K), f64(V), f64(O)
    l = None if L is None else f64(L)
    a = c = gap
    for b, (n, m) in enumerate(zip(nq, nk)):
        if only is None or b in only:
            i, j = np.arange(n)[:, None], np.arange(m)[None]
            seen = (j <= i + m - n) if causal else np.ones((n, m), dtype=bool)
            for h in range(Hq):
                g = h // (Hq // Hkv)
                kk, vv = k[c:c + m, g * D:(g + 1) * D], v[c:c + m, g * D:(g + 1) * D]
                want, lse, A, S = attend(q[a:a + n, h * D:(h + 1) * D], kk, vv, scale, seen)
                bo, bl = bounds(want, lse, A, S, vv, D, t, t)
                assert_close(o[a:a + n, h * D:(h + 1) * D], want, bo, f"sequence {b} head {h}")
                if l is not None:
                    assert_close(l[a:a + n, h], lse, bl, f"lse of sequence {b} head {h}")
        a, c = a + n, c + m
    assert np.all(o[:gap] == 7.0) and np.all(o[a:] == 7.0) and np.all(o[:, Hq * D:] == 7.0)


PROMPTS = [
    # new tokens and keys of each sequence, heads, D, type
    ([1], [1], 1, 1, 128, "bf16"),
    ([1, 2, 3, 0, 1], [1, 2, 3, 0, 1], 16, 8, 128, "bf16"),
    ([127, 128, 129], [127, 128, 129], 4, 2, 128, "f16"),
    ([255, 1, 257], [255, 1, 257], 5, 1, 128, "bf16"),
    ([40, 0, 300, 7], [168, 64, 300, 519], 6, 3, 128, "bf16"),     # earlier tokens; keys without queries
    ([200, 5, 33], [60, 0, 32], 4, 4, 128, "bf16"),                # fewer keys than queries
    ([513], [1300], 2, 1, 64, "f16"),
    ([100, 131], [100, 131], 3, 3, 80, "bf16"),
    ([70, 260], [90, 260], 4, 1, 96, "f16"),
    ([18, 150], [18, 150], 2, 2, 16, "bf16"),
    ([300], [300], 3, 1, 48, "f16"),
    ([1], [700], 8, 2, 128, "f16"),
    ([64], [3000], 10, 2, 128, "bf16"),                            # few rows, many keys
    ([3, 20], [2100, 1], 4, 1, 64, "bf16"),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D,t", PROMPTS)
def test_prompt(nq, nk, Hq, Hkv, D, t, causal):
    Q, K, V = heads(1, sum(nq), Hq, D, t, 8), heads(2, sum(nk), Hkv, D, t), heads(3, sum(nk), Hkv, D, t, 16)
    scale = 1.0 / math.sqrt(D)
    O, L = run_prompt(Q, K, V, nq, nk, Hq, Hkv, D, t, causal, scale)
    check_prompt(Q, K, V, O, L, nq, nk, Hq, Hkv, D, t, causal, scale)


@pytest.mark.parametrize("scale", [0.0, 0.02, 4.0])
def test_prompt_scales(scale):
    """Flat and peaked scores (a running maximum that keeps growing)."""
    n, Hq, Hkv, D, t = 400, 2, 1, 128, "bf16"
    Q, K, V = heads(4, n, Hq, D, t), heads(5, n, Hkv, D, t), heads(6, n, Hkv, D, t)
    K *= torch.linspace(0.1, 1.0, n, device=DEV)[:, None].to(torch.bfloat16)
    O, L = run_prompt(Q, K, V, [n], [n], Hq, Hkv, D, t, True, scale)
    O8 = O[:, :Hq * D]
    assert torch.isfinite(O8.float()).all()
    check_prompt(Q, K, V, O, L, [n], [n], Hq, Hkv, D, t, True, scale)


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_rows_of_no_sequence(causal):
    """Rows before the first and after the last sequence: NaN and infinities there reach nothing, outputs there stay."""
    nq, nk, Hq, Hkv, D, t = [60, 140], [100, 140], 4, 2, 128, "bf16"
    gap = 3
    Q, K, V = heads(7, 210, Hq, D, t), heads(8, 250, Hkv, D, t), heads(9, 250, Hkv, D, t)
    for x, n in ((Q, 200), (K, 240), (V, 240)):
        x[:gap] = float("nan")
        x[n + gap:] = float("inf")
    O, L = run_prompt(Q, K, V, nq, nk, Hq, Hkv, D, t, causal, 0.1, gap)
    check_prompt(Q, K, V, O, L, nq, nk, Hq, Hkv, D, t, causal, 0.1, gap)
    assert torch.all(L[:gap] == 7.0) and torch.all(L[200 + gap:] == 7.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_prompt_non_finite_values_stay_in_their_sequence(bad):
    nq = [100, 50, 90]
    Hq, Hkv, D, t = 2, 1, 128, "bf16"
    Q, K, V = heads(10, 240, Hq, D, t), heads(11, 240, Hkv, D, t), heads(12, 240, Hkv, D, t)
    V[100:150] = bad
    K[120:130] = bad
    for causal in (True, False):
        O, L = run_prompt(Q, K, V, nq, nq, Hq, Hkv, D, t, causal, 0.09)
        check_prompt(Q, K, V, O, L, nq, nq, Hq, Hkv, D, t, causal, 0.09, only=(0, 2))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("n,at", [(300, 270), (90, 13), (520, 400)])
def test_prompt_non_finite_values_reach_only_rows_that_see_them(n, at, bad):
    """A key and some of its values spoiled: earlier rows are right, later rows show it in those elements."""
    Hq, Hkv, D, t = 2, 1, 128, "f16"
    Q, K, V = heads(13, n, Hq, D, t), heads(14, n, Hkv, D, t), heads(15, n, Hkv, D, t)
    clean = V.clone()
    V[at, 5] = bad
    V[at, 127] = bad
    O, L = run_prompt(Q, K, V, [n], [n], Hq, Hkv, D, t, True, 0.09)
    o = O[:, :Hq * D].float().reshape(n, Hq, D)
    spoiled = o[at:, :, [5, 127]]
    assert torch.isnan(spoiled).all() if math.isnan(bad) else torch.all(spoiled == bad)
    O2, L2 = run_prompt(Q, K, clean, [n], [n], Hq, Hkv, D, t, True, 0.09)
    o2 = O2[:, :Hq * D].float().reshape(n, Hq, D)
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[at:, :, [5, 127]] = False
    assert torch.equal(o[keep], o2[keep])
    assert torch.equal(L, L2)
    # a spoiled key: rows before it do not see it
    K[at] = bad
    O3, _ = run_prompt(Q, K, clean, [n], [n], Hq, Hkv, D, t, True, 0.09)
    assert torch.equal(O3[:at], O2[:at])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("keys", [63, 64, 65, 127, 128, 129, 191, 192, 193])
def test_prompt_ends_around_half_a_tile(keys, causal):
    """Few queries against a last tile that is full, half full and one beside it;
    the rows behind the sequence's keys are not finite."""
    H, G, D = 4, 2, 128
    nq, nk = [min(keys, 33), keys, 1], [keys, keys, keys]
    Q = heads(70 + keys, sum(nq), H, D, "bf16")
    K, V = heads(80 + keys, sum(nk) + 200, G, D, "bf16"), heads(90 + keys, sum(nk) + 200, G, D, "bf16")
    K[sum(nk):] = float("nan")
    V[sum(nk):] = float("inf")
    O, L = run_prompt(Q, K, V, nq, nk, H, G, D, "bf16", causal, D ** -0.5)
    check_prompt(Q, K, V, O, L, nq, nk, H, G, D, "bf16", causal, D ** -0.5)


def test_prompt_offsets_are_clamped():
    """Offsets outside the buffers are read as the nearest end, decreasing ones as an empty sequence."""
    Hq, Hkv, D, t, n = 2, 1, 64, "bf16", 150
    Q, K, V = heads(16, n, Hq, D, t), heads(17, n, Hkv, D, t), heads(18, n, Hkv, D, t)
    ws = workspace(tb.tern_attn_prompt_workspace_bytes(2, n, n, Hq, Hkv, D))
    O = torch.full((n, Hq * D), 7.0, dtype=TYPES[t], device=DEV)
    cu = torch.tensor([-5, 60, 1 << 30], dtype=torch.int32, device=DEV)
    cu_k = torch.tensor([-9, 60, (1 << 31) - 1], dtype=torch.int32, device=DEV)
    tb.tern_attn_prompt(X[t], 2, cu, cu_k, n, n, Hq, Hkv, D, True, 0.125, Q, Hq * D, K, Hkv * D, V, Hkv * D, O, Hq * D,
                        None, ws)
    want, _ = run_prompt(Q, K, V, [60, 90], [60, 90], Hq, Hkv, D, t, True, 0.125)
    assert torch.equal(O, want[:, :Hq * D])
    O.fill_(7.0)
    cu = torch.tensor([0, 100, 40], dtype=torch.int32, device=DEV)
    tb.tern_attn_prompt(X[t], 2, cu, cu, n, n, Hq, Hkv, D, True, 0.125, Q, Hq * D, K, Hkv * D, V, Hkv * D, O, Hq * D,
                        None, ws)
    want, _ = run_prompt(Q, K, V, [100], [100], Hq, Hkv, D, t, True, 0.125)
    assert torch.equal(O[:100], want[:100, :Hq * D])
    assert torch.all(O[100:] == 7.0)
    assert tb.tern_workspace_error(ws) == 0


def test_prompt_repeats_and_streams():
    """The same call twice, on another stream, with a used workspace: the same bits."""
    nq, Hq, Hkv, D, t = [30, 700, 129], 4, 2, 128, "f16"
    n = sum(nq)
    Q, K, V = heads(19, n, Hq, D, t), heads(20, n, Hkv, D, t), heads(21, n, Hkv, D, t)
    ws = workspace(tb.tern_attn_prompt_workspace_bytes(3, n, n, Hq, Hkv, D))
    a, la = run_prompt(Q, K, V, nq, nq, Hq, Hkv, D, t, True, 0.1, ws=ws)
    torch.cuda.synchronize()
    b, lb = run_prompt(Q, K, V, nq, nq, Hq, Hkv, D, t, True, 0.1, ws=ws, stream=torch.cuda.Stream())
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_prompt_sampled_long():
    """Rows of a long prompt (past one 32-bit element of scores) against the reference."""
    n, Hq, Hkv, D, t = 5000, 10, 2, 128, "bf16"
    Q, K, V = heads(22, n, Hq, D, t), heads(23, n, Hkv, D, t), heads(24, n, Hkv, D, t)
    O, L = run_prompt(Q, K, V, [n], [n], Hq, Hkv, D, t, True, 1 / math.sqrt(D))
    rows = np.array([0, 1, 127, 128, 255, 256, 1000, 2431, 4863, 4864, 4999])
    q, k, v, o, l = f64(Q), f64(K), f64(V), f64(O), f64(L)
    for h in (0, 4, 5, 9):
        g = h // 5
        kk, vv = k[:, g * D:(g + 1) * D], v[:, g * D:(g + 1) * D]
        seen = np.arange(n)[None] <= rows[:, None]
        want, lse, A, S = attend(q[rows, h * D:(h + 1) * D], kk, vv, 1 / math.sqrt(D), seen)
        bo, bl = bounds(want, lse, A, S, vv, D, t, t)
        assert_close(o[rows, h * D:(h + 1) * D], want, bo, f"head {h}")
        assert_close(l[rows, h], lse, bl, f"lse {h}")


# ------------------------------------------------------------ single tokens

def make_cache(lens, Hkv, page, D, kind, t, seed, extra=3, spread=0.5):
    """A cache whose unused rows and pages hold NaN (codes and factors too):
    (pages, cache tensors, table, keys and values [sequence][g] in 64 bits)."""
    per = max(1, -(-max(lens) // page)) + 1
    B = len(lens)
    pages = B * per + extra
    order = np.random.default_rng(seed).permutation(pages)[:B * per].reshape(B, per)
    out, plain = [], []
    for which in range(2):
        rows = heads(seed + which, pages * page, Hkv, D, t, 0, spread).cpu()
        x = rows.reshape(pages, page, Hkv, D).transpose(1, 2).contiguous()
        used = torch.zeros((pages, page), dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(-(-n // page)):
                used[order[b, j], :min(page, n - j * page)] = True
        used = used[:, None, :]
        if kind == "x16":
            c = torch.where(used[..., None], x, torch.full((), float("nan"), dtype=x.dtype))
            value, scale = f64(x), None
        else:
            code, scale = quantise(x, kind)
            value = code_values(code, kind) * f64(scale)[..., None]
            c = torch.where(used[..., None], code, torch.full((), 0x7F, dtype=torch.uint8))   # NaN as e4m3
            scale = torch.where(used, scale, torch.full((), float("nan")))
        out.append((c, scale))
        plain.append([[value[order[b], g].reshape(-1, D)[:n] for g in range(Hkv)] for b, n in enumerate(lens)])
    table = torch.from_numpy(order.astype(np.int32))
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = [-1, 1 << 30][b % 2]        # entries past the length are never followed
    cache = [out[0][0].to(DEV), out[1][0].to(DEV)] + [None if s is None else s.to(DEV) for s in (out[0][1], out[1][1])]
    return pages, cache, table.to(DEV), plain


def run_decode(Q, lens, Hq, Hkv, D, page, kind, t, scale, pages, cache, table, ws=None, stream=None):
    B = len(lens)
    O = torch.full((B, Hq * D + 8), 7.0, dtype=TYPES[t], device=DEV)
    L = torch.full((B, Hq), 7.0, device=DEV)
    per = table.shape[1]
    ws = workspace(tb.tern_attn_decode_workspace_bytes(B, Hq, Hkv, D, per * page)) if ws is None else ws
    tb.tern_attn_decode(X[t], KV[kind], B, Hq, Hkv, D, scale, Q, Q.stride(0), pages, page, *cache, table, per,
                        torch.tensor(lens, dtype=torch.int32, device=DEV), O, O.stride(0), L, ws, stream=stream)
    if stream is not None:
        stream.synchronize()
    assert tb.tern_workspace_error(ws) == 0
    return O, L


def check_decode(Q, O, L, lens, Hq, Hkv, D, kind, t, scale, plain):
    q, o, l = f64(Q), f64(O), f64(L)
    assert np.all(o[:, Hq * D:] == 7.0)
    for b, n in enumerate(lens):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            k, v = plain[0][b][g], plain[1][b][g]
            want, lse, A, S = attend(q[b:b + 1, h * D:(h + 1) * D], k, v, scale, np.ones((1, n), dtype=bool))
            bo, bl = bounds(want, lse, A, S, v, D, t, t if kind == "x16" else "f16")
            assert_close(o[b:b + 1, h * D:(h + 1) * D], want, bo, f"sequence {b} head {h}")
            assert_close(l[b:b + 1, h], lse, bl, f"lse of sequence {b} head {h}")


DECODES = [
    # lengths, heads, D, page, type
    ([1], 1, 1, 128, 16, "bf16"),
    ([701], 40, 8, 128, 16, "bf16"),
    ([15, 16, 17, 0, 33, 31, 32], 16, 8, 128, 16, "f16"),
    ([5, 300, 0, 0, 77], 8, 1, 128, 1, "bf16"),                    # eight heads share, pages of one token
    ([1000, 3], 12, 1, 64, 4, "f16"),                              # twelve share
    ([129, 500], 16, 1, 96, 64, "bf16"),
    ([260], 40, 2, 128, 32, "f16"),                                # twenty share: more than one pass of sixteen
    ([90, 257, 2], 6, 6, 80, 8, "bf16"),
    ([400], 3, 1, 16, 128, "bf16"),
    ([64, 65], 4, 2, 48, 512, "f16"),
    ([0, 0], 4, 2, 128, 16, "bf16"),
    ([4100, 1, 2050], 10, 2, 128, 16, "bf16"),
]


@pytest.mark.parametrize("kind", ["x16", "e4m3", "i8"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page,t", DECODES)
def test_decode(lens, Hq, Hkv, D, page, t, kind):
    Q = heads(31, len(lens), Hq, D, t, 8)
    pages, cache, table, plain = make_cache(lens, Hkv, page, D, kind, t, 32)
    scale = 1.0 / math.sqrt(D)
    O, L = run_decode(Q, lens, Hq, Hkv, D, page, kind, t, scale, pages, cache, table)
    check_decode(Q, O, L, lens, Hq, Hkv, D, kind, t, scale, plain)


@pytest.mark.parametrize("kind", ["x16", "e4m3", "i8"])
@pytest.mark.parametrize("scale", [0.0, 0.02, 3.0])
def test_decode_scales(scale, kind):
    lens, Hq, Hkv, D, page, t = [900, 40], 5, 1, 128, 16, "f16"
    Q = heads(33, 2, Hq, D, t)
    pages, cache, table, plain = make_cache(lens, Hkv, page, D, kind, t, 34)
    O, L = run_decode(Q, lens, Hq, Hkv, D, page, kind, t, scale, pages, cache, table)
    check_decode(Q, O, L, lens, Hq, Hkv, D, kind, t, scale, plain)


# Batches whose work is dealt to the SMs in each way: several whole items per CTA,
# some CTAs short of one, with empty sequences between them; an item or part of one
# per CTA; unequal lengths cut by weight, with more items than CTAs and with fewer.
BATCHES = [
    [33] * 50,
    [40, 0, 33, 37, 0, 0, 48] * 11 + [0, 35],
    [200] * 18,
    [180, 200, 190, 0] * 10,
    [1700] + [20, 50, 5] * 20,
    [2500, 3, 40, 700, 0, 90],
]


@pytest.mark.parametrize("kind", ["x16", "e4m3", "i8"])
@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_decode_batches(batch, kind):
    lens, Hq, Hkv, D = BATCHES[batch], 16, 8, 128
    Q = heads(131, len(lens), Hq, D, "bf16", 8)
    pages, cache, table, plain = make_cache(lens, Hkv, 16, D, kind, "bf16", 132)
    scale = 1.0 / math.sqrt(D)
    ws = workspace(tb.tern_attn_decode_workspace_bytes(len(lens), Hq, Hkv, D, table.shape[1] * 16))
    for _ in range(2):   # the second call finds the workspace as the first left it
        O, L = run_decode(Q, lens, Hq, Hkv, D, 16, kind, "bf16", scale, pages, cache, table, ws=ws)
    check_decode(Q, O, L, lens, Hq, Hkv, D, kind, "bf16", scale, plain)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 40])
def test_decode_factors_of_any_size(size, kind):
    """Values, keys and queries far outside fp16's range: codes stay exact and the factors are fp32."""
    lens, Hq, Hkv, D, page, t = [200], 4, 2, 64, 16, "bf16"
    Q = heads(35, 1, Hq, D, t)
    pages, cache, table, plain = make_cache(lens, Hkv, page, D, kind, t, 36)
    cache[2] *= 1.0 / size                        # keys
    cache[3] *= size                              # values
    Q *= size
    plain = [[[k / size for k in s] for s in plain[0]], [[v * size for v in s] for s in plain[1]]]
    O, L = run_decode(Q, lens, Hq, Hkv, D, page, kind, t, 0.125, pages, cache, table)
    O = O.double()
    O[:, :Hq * D] /= size
    plain[1] = [[v / size for v in s] for s in plain[1]]
    check_decode(Q, O, L, lens, Hq, Hkv, D, kind, t, 0.125, plain)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_decode_values_of_unequal_size(kind):
    """Value factors that grow and shrink by 2^24 along a sequence."""
    lens, Hq, Hkv, D, page, t = [640], 3, 1, 128, 16, "bf16"
    Q = heads(37, 1, Hq, D, t)
    pages, cache, table, plain = make_cache(lens, Hkv, page, D, kind, t, 38)
    steps = 2.0 ** np.round(24 * np.sin(np.arange(640) / 50.0))
    for j in range(640):
        cache[3][int(table[0, j // page]), 0, j % page] *= float(steps[j])
    plain[1] = [[v * steps[:, None] for v in s] for s in plain[1]]
    O, L = run_decode(Q, lens, Hq, Hkv, D, page, kind, t, 0.09, pages, cache, table)
    check_decode(Q, O, L, lens, Hq, Hkv, D, kind, t, 0.09, plain)


def test_decode_hidden_pages_and_lengths():
    """A page id outside the cache hides its tokens; lengths are clamped to the table."""
    Hq, Hkv, D, page, t = 4, 2, 128, 16, "bf16"
    lens = [100, 80]
    Q = heads(39, 2, Hq, D, t)
    pages, cache, table, plain = make_cache(lens, Hkv, page, D, "x16", t, 40)
    table[0, 2] = pages
    table[1, 0] = -7
    O, L = run_decode(Q, lens, Hq, Hkv, D, page, "x16", t, 0.1, pages, cache, table)
    for part in plain:
        part[0] = [np.delete(x, np.s_[32:48], 0) for x in part[0]]
        part[1] = [x[16:] for x in part[1]]
    check_decode(Q, O, L, [84, 64], Hq, Hkv, D, "x16", t, 0.1, plain)
    # lengths beyond the table and below zero
    lens = [96, 40]
    pages, cache, table, plain = make_cache(lens, Hkv, page, D, "x16", t, 41)
    table = table[:, :6].contiguous()
    O, L = run_decode(Q, [5000, -3], Hq, Hkv, D, page, "x16", t, 0.1, pages, cache, table)
    plain = [[p[0], [x[:0] for x in p[1]]] for p in plain]
    check_decode(Q, O, L, [96, 0], Hq, Hkv, D, "x16", t, 0.1, plain)


def test_decode_repeats_and_streams():
    """One workspace over calls of several shapes, and another stream: the same bits."""
    Hq, Hkv, D, page, t = 10, 2, 128, 16, "bf16"
    ws = workspace(tb.tern_attn_decode_workspace_bytes(40, Hq, Hkv, D, 6000))
    seen = {}
    for turn in range(2):
        for lens in ([5000], [33] * 40, [7, 2000, 0]):
            Q = heads(42, len(lens), Hq, D, t)
            pages, cache, table, plain = make_cache(lens, Hkv, page, D, "e4m3", t, 43)
            torch.cuda.synchronize()
            O, L = run_decode(Q, lens, Hq, Hkv, D, page, "e4m3", t, 0.1, pages, cache, table, ws,
                              torch.cuda.Stream() if turn else None)
            key = tuple(lens)
            if key in seen:
                assert torch.equal(O, seen[key][0]) and torch.equal(L, seen[key][1])
            else:
                check_decode(Q, O, L, lens, Hq, Hkv, D, "e4m3", t, 0.1, plain)
            seen[key] = (O, L)


def test_decode_offsets_past_32_bits():
    """Pages beyond 2^32 bytes of codes."""
    Hq, Hkv, D, page, t = 8, 8, 128, 64, "bf16"
    pages = (1 << 32) // (Hkv * D * page) + 2
    small_pages, small, table, plain = make_cache([150], Hkv, page, D, "i8", t, 44, extra=0)
    big = [torch.zeros((pages,) + x.shape[1:], dtype=x.dtype, device=DEV) for x in small]
    shift = pages - small_pages
    for x, y in zip(big, small):
        x[shift:] = y
    table = torch.where((table >= 0) & (table < small_pages), table + shift, table)
    Q = heads(45, 1, Hq, D, t)
    O, L = run_decode(Q, [150], Hq, Hkv, D, page, "i8", t, 0.1, pages, big, table)
    check_decode(Q, O, L, [150], Hq, Hkv, D, "i8", t, 0.1, plain)


def test_decode_equals_prompt_of_one_token():
    """A single token over a 16-bit cache is a prompt of one row (within the bounds of both)."""
    n, Hq, Hkv, D, page, t = 333, 8, 2, 128, 16, "bf16"
    Q = heads(46, 1, Hq, D, t)
    pages, cache, table, plain = make_cache([n], Hkv, page, D, "x16", t, 47)
    O, L = run_decode(Q, [n], Hq, Hkv, D, page, "x16", t, 0.1, pages, cache, table)
    slots = torch.tensor([int(table[0, j // page]) * page + j % page for j in range(n)], device=DEV)
    K, V = (torch.empty((n, Hkv * D), dtype=TYPES[t], device=DEV) for _ in range(2))
    tb.tern_kv_read(X[t], KV["x16"], n, Hkv, D, slots, pages, page, *cache, K, Hkv * D, V, Hkv * D)
    P, M = run_prompt(Q, K, V, [1], [n], Hq, Hkv, D, t, True, 0.1)
    check_prompt(Q, K, V, P, M, [1], [n], Hq, Hkv, D, t, True, 0.1)
    check_decode(Q, O, L, [n], Hq, Hkv, D, "x16", t, 0.1, plain)
