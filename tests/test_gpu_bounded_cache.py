"""The norm, the int8 linear, the cache and what keeps it within a budget, run together as a
decoder layer runs them, over many steps, against the same layer in 64 bits.

The reference keeps its own cache of the tokens that the calls report as kept: which tokens
those are is checked for itself (the choice is exact for the weights that the calls hold, and
those are within their bound of the reference's), so that a choice between two nearly equal
weights does not decide the comparison.

Tolerance (relative 2-norm of a step's output).  Codes of the normalised input: half a step of
a / 127 uniformly distributed, with the largest of 1024 normal values about 3.5 standard deviations
3.5 / 127 / sqrt(12) = 0.008, through the linear as it is; keys, values and queries rounded to
bf16 2^-9 rms each; attention weights and outputs to bf16 likewise; the second rounding of the
stream.  The sum is below 0.02."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import f64, randn  # noqa: E402
from budget_util import keep_reference  # noqa: E402
from gpu_util import DEV  # noqa: E402
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402

pytestmark = pytest.mark.gpu

HIDDEN, HQ, HKV, D, PAGE = 1024, 16, 8, 128, 16
BUDGET, FIRST, RECENT = 48, 4, 16
BF16 = tb.TERN_OUT_BF16


def ternary(seed, n, k):
    """Tiled weights and the same in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(-1, 2, (n, k), generator=g, dtype=torch.int8)
    scales = torch.exp(0.3 * torch.randn((n, k // 128), generator=g) - 4).to(torch.float16)
    packed = torch.empty((n, k // 4), dtype=torch.uint8, device=DEV)
    tb.tern_pack(t.to(DEV), n, k, packed)
    tiled = torch.empty(tb.tern_tiled_bytes(n, k), dtype=torch.uint8, device=DEV)
    tb.tern_repack(packed, scales.view(torch.int16).to(DEV), n, k, tiled)
    return tiled, f64(t) * f64(scales).repeat(128, axis=1)


def norm(x, w):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * w


@pytest.mark.parametrize("B,steps", [(1, 70), (3, 60)])
def test_steps_over_a_bounded_cache(B, steps):
    N = (HQ + 2 * HKV) * D
    qkv_tiled, qkv_dense = ternary(1, N, HIDDEN)
    w_in = (1 + 0.1 * randn(3, HIDDEN)).to(torch.bfloat16)
    w_head = (0.1 * randn(4, D)).to(torch.bfloat16)           # about zero: w_add = 1
    stream = torch.zeros((B, HIDDEN), dtype=torch.bfloat16, device=DEV)
    per = (BUDGET + PAGE) // PAGE + 1
    pages = B * per
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).to(torch.int32).reshape(B, per).to(DEV)
    k_cache, v_cache = (torch.zeros((pages, HKV, PAGE, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    weight = torch.full((pages, HKV, PAGE), float("nan"), device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    new_lens, keep = torch.empty_like(lens), torch.empty((B, HKV, BUDGET), dtype=torch.int32, device=DEV)
    xq, a = torch.empty(tb.tern_xq_bytes(B, HIDDEN), dtype=torch.int8, device=DEV), torch.empty(B, device=DEV)
    qkv = torch.empty((B, N), dtype=torch.bfloat16, device=DEV)
    o, lse = torch.empty((B, HQ * D), dtype=torch.bfloat16, device=DEV), torch.empty((B, HQ), device=DEV)
    ws_lin = torch.zeros(tb.tern_i8_workspace_bytes(B, N, HIDDEN), dtype=torch.uint8, device=DEV)
    ws_att = torch.zeros(tb.tern_attn_decode_workspace_bytes(B, HQ, HKV, D, per * PAGE), dtype=torch.uint8, device=DEV)
    freq, amp = tb.tern_rope_freqs(D, 1e6)
    freq_dev = torch.tensor(freq, dtype=torch.float32, device=DEV)

    # the reference: stream, and for each (sequence, head) keys, values and weights of its tokens
    s64 = np.zeros((B, HIDDEN))
    cache = [[[np.zeros((0, D)), np.zeros((0, D)), np.zeros(0)] for _ in range(HKV)] for _ in range(B)]
    freq64 = np.asarray(freq, dtype=np.float64)
    wi, wh = f64(w_in), f64(w_head) + 1

    for step in range(steps):
        x = randn(100 + step, B, HIDDEN)
        tb.tern_rms_norm_i8(0, tb.TERN_OUT_F32, B, HIDDEN, x.to(DEV), HIDDEN, BF16, stream, HIDDEN, stream, HIDDEN, w_in.to(DEV),
                            0.0, 1e-6, xq, a)
        tb.tern_linear_i8(xq, a, qkv_tiled, B, N, HIDDEN, qkv, N, BF16, ws_lin)
        # queries and keys head by head, in place in the projection's output
        tb.tern_rms_norm(0, BF16, B, HQ + HKV, D, qkv, N, BF16, None, 0, None, 0, w_head.to(DEV), 1.0, 1e-6, qkv, N)
        pos = torch.full((B,), step, dtype=torch.int32, device=DEV)
        slots = table[torch.arange(B, device=DEV), (lens // PAGE).long()].long() * PAGE + (lens % PAGE).long()
        q = torch.empty((B, HQ * D), dtype=torch.bfloat16, device=DEV)
        tb.tern_rope_kv_write(0, tb.TERN_KV_X16, 0, B, HQ, HKV, D, D, pos, freq_dev, amp, qkv, N, q, HQ * D, qkv[:, HQ * D:], N,
                              qkv[:, (HQ + HKV) * D:], N, slots, pages, PAGE, k_cache, v_cache)
        known = lens.clone()
        lens += 1
        tb.tern_attn_decode(0, tb.TERN_KV_X16, B, HQ, HKV, D, D ** -0.5, q, HQ * D, pages, PAGE, k_cache, v_cache, None, None,
                            table, per, lens, o, HQ * D, lse, ws_att)
        tb.tern_attn_weights(0, tb.TERN_KV_X16, B, None, B, HQ, HKV, D, D ** -0.5, q, HQ * D, lse, pages, PAGE, k_cache, None,
                             table, per, lens, known, 0.9, weight)
        before = weight[table.long()].transpose(1, 2).reshape(B, HKV, -1).cpu().numpy()
        tb.tern_kv_keep(B, HKV, pages, PAGE, weight, table, per, lens, BUDGET, FIRST, RECENT, keep, new_lens)
        tb.tern_kv_compact(tb.TERN_KV_X16, B, HKV, D, pages, PAGE, k_cache, v_cache, None, None, weight, table, per, keep, BUDGET)
        n = int(lens[0])
        lens.copy_(new_lens)

        # the same in 64 bits
        s64 = s64 + f64(x)
        y = norm(s64, wi) @ qkv_dense.T
        heads = y.reshape(B, HQ + 2 * HKV, D)
        qk = norm(heads[:, :HQ + HKV], wh)
        angle = step * freq64
        c, s = np.cos(angle), np.sin(angle)
        lo, hi = qk[..., :D // 2], qk[..., D // 2:]
        qk = np.concatenate([lo * c - hi * s, hi * c + lo * s], -1)
        lists = keep.cpu().numpy()
        assert new_lens.tolist() == [min(n, BUDGET)] * B
        out = np.zeros((B, HQ, D))
        for b in range(B):
            for g in range(HKV):
                mine = cache[b][g]
                mine[0] = np.concatenate([mine[0], qk[b, HQ + g][None]])
                mine[1] = np.concatenate([mine[1], heads[b, HQ + HKV + g][None]])
                z = qk[b, 2 * g:2 * g + 2] @ mine[0].T * D ** -0.5
                p = np.exp(z - z.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                out[b, 2 * g:2 * g + 2] = p @ mine[1]
                mine[2] = 0.9 * np.concatenate([mine[2], [0.0]]) + p.sum(0)
                # weights: the scores' error (inputs off by 0.02 at most, scores of a few units) moves them
                # by less than a tenth of themselves
                assert np.all(np.abs(before[b, g, :n] - mine[2]) <= 0.1 * mine[2] + 1e-4), (step, b, g)
                got = lists[b, g][lists[b, g] >= 0]
                assert np.array_equal(got, keep_reference(before[b, g, :n], n, BUDGET, FIRST, RECENT))
                for i in range(3):
                    mine[i] = mine[i][got]
        err = np.linalg.norm(f64(o).reshape(B, HQ, D) - out) / np.linalg.norm(out)
        assert err <= 0.02, (step, err)
    assert lens.tolist() == [min(steps, BUDGET)] * B
    err = np.linalg.norm(f64(stream) - s64) / np.linalg.norm(s64)
    assert err <= 2.0 ** -8 * np.sqrt(steps)


def test_example_with_norm_and_budget():
    """The example runs with both; with the norm alone its check holds as without (the norm's own roundings are two
    more of the input's size)."""
    import os
    import sys
    from conftest import ROOT
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import attention_block
    lines = []
    assert attention_block.run(seqs=2, prompt=330, part=200, steps=3, cache="i8", out=lines.append, norm=True) <= 2.5 * 0.01 + 0.01
    assert attention_block.run(seqs=2, prompt=130, part=100, steps=4, cache="e4m3", out=lines.append, norm=True, budget=64) is None
    assert lines[-1] == "tokens kept: [64, 64] of 134"
