"""Attention results do not depend on what ran before them."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import heads  # noqa: E402
from test_gpu_attention import run_prompt  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nq,nk,Hq,Hkv,D,t", [
    ([64], [3000], 10, 2, 128, "bf16"),             # tiles of 5 heads x 25 tokens: three rows of 128 are no one's
    ([640, 600, 17], [640, 900, 80], 24, 4, 64, "f16"),
    ([30, 129, 61], [30, 129, 400], 6, 2, 128, "bf16"),
])
def test_prompt_bits_do_not_depend_on_the_call_before(nq, nk, Hq, Hkv, D, t):
    """Shared memory holds outputs or queries of the call before, of as many rows as fill
    every tile: large ones, then small ones."""
    Q, K, V = heads(1, sum(nq), Hq, D, t), heads(2, sum(nk), Hkv, D, t), heads(3, sum(nk), Hkv, D, t)
    n = 2048
    big = [heads(4 + i, n, 8, D, t) for i in range(3)]
    big[0] *= 30.0
    big[2] *= 300.0
    small = [heads(7 + i, n, 8, D, t) for i in range(3)]
    small[0] *= 0.001
    small[2] *= 0.001
    results = []
    for other in (big, small, big):
        run_prompt(*other, [n], [n], 8, 8, D, t, True, 1.0)
        run_prompt(*[x[:120 * 40] for x in other], [40] * 51, [40] * 51, 8, 8, D, t, True, 1.0)
        results.append(run_prompt(Q, K, V, nq, nk, Hq, Hkv, D, t, False, D ** -0.5))
    for O, L in results[1:]:
        assert torch.equal(O, results[0][0]) and torch.equal(L, results[0][1])
