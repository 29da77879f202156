"""Prompt attention directly before kernels that hold tensor memory while they wait
for it: the streaming linear, the GEMM and prompt attention itself, in chains long
enough that launches overlap."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gpu_util import DEV  # noqa: E402
from test_gpu_workspace import linear_call, prompt_call, ternary  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nq,nk", [([9, 7], [9, 7]), ([64], [3000]), ([700, 800], [700, 900])])
@pytest.mark.parametrize("M", [1, 4, 48])
def test_prompt_then_linear(M, nq, nk, D):
    attend = prompt_call(nq, nk, 8, 2, D, "bf16")
    linear = linear_call(M, 640, 1280, ternary(640, 1280, 30))
    want = [[y.clone() for y in call(torch.zeros(n, dtype=torch.uint8, device=DEV))] for n, call in (attend, linear)]
    ws = torch.zeros(max(attend[0], linear[0]), dtype=torch.uint8, device=DEV)
    got = []
    for _ in range(20):
        got.append((attend[1](ws), linear[1](ws)))
    for pair in got:
        for x, y in zip(pair, want):
            assert all(torch.equal(u, v) for u, v in zip(x, y))
