"""One workspace under calls of every kind in turn.

A zeroed workspace serves any sequence of calls on one stream: what a call
leaves in it (partial sums, converted activations, partial attention results)
reaches no later one.  Every call is made once with a workspace of its own and
then, on one shared by all, directly after every call; outputs are equal bit
for bit, since each call is deterministic."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import heads  # noqa: E402
from gpu_util import DEV, tiled_from_ternary  # noqa: E402
from test_gpu_attention import KV, TYPES, X, cumulative, make_cache  # noqa: E402
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402

pytestmark = pytest.mark.gpu


def prompt_call(nq, nk, Hq, Hkv, D, t):
    Tq, Tkv, B = sum(nq), sum(nk), len(nq)
    Q, K, V = heads(1, Tq, Hq, D, t), heads(2, Tkv, Hkv, D, t), heads(3, Tkv, Hkv, D, t)
    cu_q, cu_k = cumulative(nq).to(DEV), cumulative(nk).to(DEV)

    def call(ws):
        O = torch.full((Tq, Hq * D), 7.0, dtype=TYPES[t], device=DEV)
        L = torch.full((Tq, Hq), 7.0, device=DEV)
        tb.tern_attn_prompt(X[t], B, cu_q, cu_k, Tq, Tkv, Hq, Hkv, D, True, 0.1, Q, Hq * D, K, Hkv * D, V, Hkv * D, O,
                            Hq * D, L, ws)
        return O, L
    return tb.tern_attn_prompt_workspace_bytes(B, Tq, Tkv, Hq, Hkv, D), call


def decode_call(lens, Hq, Hkv, D, kind, t):
    B = len(lens)
    Q = heads(4, B, Hq, D, t)
    pages, cache, table, _ = make_cache(lens, Hkv, 16, D, kind, t, 5)
    per, n = table.shape[1], torch.tensor(lens, dtype=torch.int32, device=DEV)

    def call(ws):
        O = torch.full((B, Hq * D), 7.0, dtype=TYPES[t], device=DEV)
        L = torch.full((B, Hq), 7.0, device=DEV)
        tb.tern_attn_decode(X[t], KV[kind], B, Hq, Hkv, D, 0.1, Q, Hq * D, pages, 16, *cache, table, per, n, O, Hq * D, L, ws)
        return O, L
    return tb.tern_attn_decode_workspace_bytes(B, Hq, Hkv, D, per * 16), call


def ternary(N, K, seed):
    rng = np.random.default_rng(seed)
    t = rng.integers(-1, 2, (N, K)).astype(np.int8)
    s = (0.01 + 0.02 * rng.random((N, K // 128))).astype(np.float16).view(np.uint16)
    return tiled_from_ternary(t, s)


def linear_call(M, N, K, tiled):
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)

    def call(ws):
        Y = torch.full((M, N), 7.0, device=DEV)
        tb.tern_linear(x, K, tiled, M, N, K, Y, N, ws)
        return (Y,)
    return tb.tern_workspace_bytes(M, N, K), call


def grouped_call(M, Ns, Ks):
    tiled = [ternary(n, k, 20 + i) for i, (n, k) in enumerate(zip(Ns, Ks))]
    xs = [torch.randn((M, k), generator=torch.Generator().manual_seed(k)).to(torch.bfloat16).to(DEV) for k in Ks]

    def call(ws):
        Ys = [torch.full((M, n), 7.0, device=DEV) for n in Ns]
        tb.tern_linear_grouped(tb.TERN_X_BF16, M, xs, list(Ks), tiled, list(Ns), list(Ks), Ys, list(Ns), tb.TERN_OUT_F32, ws)
        return Ys
    return tb.tern_grouped_workspace_bytes(M, list(Ns), list(Ks)), call


def i8_call(M, N, K, tiled):
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).to(DEV)
    xq = torch.empty(tb.tern_xq_bytes(M, K), dtype=torch.int8, device=DEV)
    a = torch.empty(M, device=DEV)
    tb.tern_quantize_x(x, tb.TERN_X_BF16, K, M, K, xq, a)

    def call(ws):
        Y = torch.full((M, N), 7.0, device=DEV)
        tb.tern_linear_i8(xq, a, tiled, M, N, K, Y, N, tb.TERN_OUT_F32, ws)
        return (Y,)
    return tb.tern_i8_workspace_bytes(M, N, K), call


def all_calls():
    N, K = 640, 5120
    w = ternary(N, K, 8)
    return {
        "prompt, keys split, 5 parts": prompt_call([64], [3000], 10, 2, 128, "bf16"),
        "prompt, keys split, short rows": prompt_call([3, 20], [2100, 1], 4, 1, 64, "bf16"),
        "prompt, one pass": prompt_call([30, 129], [30, 129], 4, 2, 128, "bf16"),
        # grids of 20, of 80 and of all SMs; items split in each
        "decode, few CTAs": decode_call([300], 2, 1, 128, "e4m3", "bf16"),
        "decode, more CTAs": decode_call([1300, 0, 700], 10, 2, 128, "x16", "bf16"),
        "decode, all SMs": decode_call([9000, 5, 4000, 0, 1700], 16, 8, 128, "i8", "bf16"),
        "linear of one token": linear_call(1, N, K, w),
        "linear of 4 tokens": linear_call(4, N, K, w),
        "linear of 40 tokens": linear_call(40, N, K, w),
        "linear of many rows": linear_call(2, 128 * 400, 256, ternary(128 * 400, 256, 9)),
        "grouped linears": grouped_call(3, [384, 1000], [2560, 1280]),
        "int8 linear": i8_call(2, N, K, w),
    }


def test_one_workspace_serves_every_sequence_of_calls():
    calls = all_calls()
    torch.cuda.synchronize()
    alone = {k: [y.clone() for y in call(torch.zeros(n, dtype=torch.uint8, device=DEV))] for k, (n, call) in calls.items()}
    shared = torch.zeros(max(n for n, _ in calls.values()), dtype=torch.uint8, device=DEV)
    wrong = []
    for first in calls:
        for second in calls:
            calls[first][1](shared)
            got = calls[second][1](shared)
            if not all(torch.equal(x, y) for x, y in zip(got, alone[second])):
                wrong.append((first, second))
    assert tb.tern_workspace_error(shared) == 0
    assert not wrong, f"{len(wrong)} of {len(calls) ** 2}: {wrong[:6]}"


def test_workspaces_of_one_size_serve_shapes_that_need_less():
    """Calls of shrinking and growing shapes on the largest one's workspace."""
    shapes = [decode_call([n], 16, 8, 128, "e4m3", "bf16") for n in (100, 900, 3000, 9000)]
    torch.cuda.synchronize()
    alone = [[y.clone() for y in call(torch.zeros(n, dtype=torch.uint8, device=DEV))] for n, call in shapes]
    shared = torch.zeros(max(n for n, _ in shapes), dtype=torch.uint8, device=DEV)
    for order in ((0, 1, 2, 3), (3, 2, 1, 0), (0, 3, 0, 2, 1, 3)):
        for i in order:
            got = shapes[i][1](shared)
            assert all(torch.equal(x, y) for x, y in zip(got, alone[i])), (order, i)
