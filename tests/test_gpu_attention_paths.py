"""Shapes that take the attention kernels' other ways to the same answer (bounds:
attn_util.py): two tiles per CTA without split keys, for several sequences;
batches of more sequences than a warp has lanes; the 64-bit arithmetic that
deals single tokens out under a wide page table."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import heads  # noqa: E402
from gpu_util import DEV  # noqa: E402
from test_gpu_attention import check_decode, check_prompt, make_cache, run_decode, run_prompt  # noqa: E402

pytestmark = pytest.mark.gpu

# Enough keys and blocks for two tiles per CTA and no split, ragged.
TWO_TILES = [
    ([640, 600, 17], [640, 900, 80], 32, 4, 128),
    ([900, 0, 1700, 1, 1900], [900, 3, 1900, 40, 2100], 8, 8, 64),
    ([700, 900, 1000], [700, 900, 1100], 16, 8, 96),
]


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D", TWO_TILES)
def test_prompt_two_tiles(nq, nk, Hq, Hkv, D, causal, t):
    Q, K, V = heads(1, sum(nq), Hq, D, t, 8), heads(2, sum(nk), Hkv, D, t), heads(3, sum(nk), Hkv, D, t, 16)
    scale = 1.0 / math.sqrt(D)
    O, L = run_prompt(Q, K, V, nq, nk, Hq, Hkv, D, t, causal, scale)
    check_prompt(Q, K, V, O, L, nq, nk, Hq, Hkv, D, t, causal, scale)


# Unsplit (several sequences, one) and with the keys split over CTAs.
SPOILED = [([700, 900, 1000], 16, 8, 128), ([800], 2, 1, 128), ([3000], 4, 2, 64)]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("n,Hq,Hkv,D", SPOILED)
def test_prompt_two_tiles_non_finite_values(n, Hq, Hkv, D, bad):
    """Two values of each sequence spoiled: rows before them are as they were, rows from
    them on show them in those elements, the other sequences nothing."""
    t, rows = "f16", sum(n)
    Q, K, V = heads(4, rows, Hq, D, t), heads(5, rows, Hkv, D, t), heads(6, rows, Hkv, D, t)
    O2, L2 = run_prompt(Q, K, V, n, n, Hq, Hkv, D, t, True, 0.09)
    spoiled = torch.zeros((rows, Hq, D), dtype=torch.bool, device=DEV)
    a = 0
    for b, m in enumerate(n):
        at = [m // 3, m - 5, 1][b % 3]
        V[a + at].reshape(Hkv, D)[:, [3, D - 2]] = bad
        spoiled[a + at:a + m, :, [3, D - 2]] = True
        a += m
    O, L = run_prompt(Q, K, V, n, n, Hq, Hkv, D, t, True, 0.09)
    o, o2 = (x[:, :Hq * D].float().reshape(rows, Hq, D) for x in (O, O2))
    # (a weight below 2^-24 of the largest is zero in fp16, and zero times infinity NaN)
    assert not torch.isfinite(o[spoiled]).any()
    assert torch.equal(o[~spoiled], o2[~spoiled])
    assert torch.equal(L, L2)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B", [33, 64, 65, 128, 129, 300])
def test_prompt_many_sequences(B, causal, t):
    """Batches past 32, 64 and 128 sequences, empty ones among them."""
    nq = [(7 * b) % 41 if b % 5 else 0 for b in range(B)]
    nk = [n + (b % 3) * 20 for b, n in enumerate(nq)]
    nq[-1], nk[-1] = 130, 200
    Hq, Hkv, D = 4, 2, 128
    Q, K, V = heads(7, sum(nq), Hq, D, t), heads(8, sum(nk), Hkv, D, t), heads(9, sum(nk), Hkv, D, t)
    O, L = run_prompt(Q, K, V, nq, nk, Hq, Hkv, D, t, causal, 0.1)
    check_prompt(Q, K, V, O, L, nq, nk, Hq, Hkv, D, t, causal, 0.1)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B", [40, 70])
def test_prompt_many_sequences_two_tiles(B, causal):
    """The two-tile form finds its sequences 32 at a time."""
    nq = [300 if b % 4 else 0 for b in range(B)]
    nk = [n + 900 for n in nq]
    Hq, Hkv, D, t = 2, 2, 64, "bf16"
    Q, K, V = heads(10, sum(nq), Hq, D, t), heads(11, sum(nk), Hkv, D, t), heads(12, sum(nk), Hkv, D, t)
    O, L = run_prompt(Q, K, V, nq, nk, Hq, Hkv, D, t, causal, 0.125)
    check_prompt(Q, K, V, O, L, nq, nk, Hq, Hkv, D, t, causal, 0.125)


# Lengths whose work is dealt whole (several items per CTA, CTAs per item) and by weight.
WIDE = [[33] * 64, [40, 0, 33, 37] * 16, [600] + [20, 50, 5] * 21, [1500, 3, 40, 700, 0, 90] + [0] * 58, [0] * 64]


@pytest.mark.parametrize("kind", ["x16", "e4m3", "i8"])
@pytest.mark.parametrize("batch", range(len(WIDE)))
def test_decode_wide_page_table(batch, kind):
    """A page table for 2^20 tokens per sequence, of which the lengths use few: the
    largest product of the dealing's arithmetic passes 2^31."""
    lens, Hq, Hkv, D, page, t = WIDE[batch], 16, 8, 128, 16, "bf16"
    Q = heads(13, len(lens), Hq, D, t)
    pages, cache, table, plain = make_cache(lens, Hkv, page, D, kind, t, 14)
    wide = torch.full((len(lens), (1 << 20) // page), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    scale = 1.0 / math.sqrt(D)
    O, L = run_decode(Q, lens, Hq, Hkv, D, page, kind, t, scale, pages, cache, wide)
    check_decode(Q, O, L, lens, Hq, Hkv, D, kind, t, scale, plain)
    N, M = run_decode(Q, lens, Hq, Hkv, D, page, kind, t, scale, pages, cache, table)   # 32-bit dealing
    check_decode(Q, N, M, lens, Hq, Hkv, D, kind, t, scale, plain)
