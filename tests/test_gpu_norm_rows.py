"""Norms of long rows where there are many: each CTA with several runs of a row to a thread,
in CTAs of any number of warps.  References and bounds are those of test_gpu_norm.py, whose
thread adds 32 squares at most here too."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import TYPES, f64  # noqa: E402
from gpu_util import DEV  # noqa: E402
from test_gpu_norm import DTYPE, E, ELEM, STEP, X16, close, inputs, padded, reference, y_bound  # noqa: E402
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402

pytestmark = pytest.mark.gpu


def many(change):
    return 4 * torch.cuda.get_device_properties(0).multi_processor_count + change


@pytest.mark.parametrize("change", [-1, 0, 3])
@pytest.mark.parametrize("K", [1032, 1152, 5120, 8200, 16392])
@pytest.mark.parametrize("t,inp,res", [("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"), ("f16", "f32", "f32"), ("bf16", "f32", "bf16"),
                                       ("f16", "f16", None), ("bf16", "f32", None)])
def test_norm_of_many_long_rows(change, K, t, inp, res):
    T = many(change)
    x, r, w = inputs(K + change, T, K, inp, res, K, t)
    X, R = padded(x, 8), None if r is None else padded(r, 16)
    S = None if r is None else torch.full((T, K + 24), 7.0, dtype=DTYPE[res], device=DEV)
    Y = torch.full((T, K + 8), 7.0, dtype=TYPES[t], device=DEV)
    tb.tern_rms_norm(X16[t], ELEM[inp], T, 1, K, X, K + 8, ELEM[res or "f32"], R, K + 16, S, K + 24, w.to(DEV), 0.5, 1e-6, Y, K + 8)
    s, y = reference(x, r, w, 0.5, 1e-6, 1)
    close(Y[:, :K], y, y_bound(y, t), "y")
    assert (Y[:, K:] == 7.0).all()
    if S is not None:
        close(S[:, :K], s, abs(s) * (STEP[res] + 2.0 ** -23) + 2.0 ** -25, "s")
        assert (S[:, K:] == 7.0).all()


@pytest.mark.parametrize("change", [-1, 0, 3])
@pytest.mark.parametrize("K", [1152, 5120, 8320, 16512])
@pytest.mark.parametrize("t,inp,res", [("bf16", "f32", "bf16"), ("f16", "f16", None), ("bf16", "bf16", "f32")])
def test_codes_of_many_long_rows(change, K, t, inp, res):
    M = many(change)
    x, r, w = inputs(K + change, M, K, inp, res, K, t)
    S = None if r is None else torch.empty((M, K), dtype=DTYPE[res], device=DEV)
    q = torch.full((M, K), 99, dtype=torch.int8, device=DEV)
    a = torch.empty((M,), device=DEV)
    tb.tern_rms_norm_i8(X16[t], ELEM[inp], M, K, x.to(DEV), K, ELEM[res or "f32"], None if r is None else r.to(DEV), K, S, K,
                        w.to(DEV), 0.0, 1e-5, q, a)
    s, y = reference(x, r, w, 0.0, 1e-5, 1)
    want_a = abs(y).max(1) / 127
    close(a, want_a, want_a * E, "a")
    code = f64(q).reshape(M, K // 16, 2, 8).swapaxes(2, 3).reshape(M, K)
    assert (abs(code - y / want_a[:, None]) <= 0.5 + 254 * E).all()
    if S is not None:
        close(S, s, abs(s) * (STEP[res] + 2.0 ** -23) + 2.0 ** -25, "s")


@pytest.mark.parametrize("K", [64, 1024, 5120])
def test_in_the_streams_place(K):
    """The normalised rows over the residual stream, by the same type and leading dimension; the sum over the input or not wanted."""
    T = many(3)
    x, r, w = inputs(K, T, K, "bf16", "bf16", K, "bf16")
    s, y = reference(x, r, w, 0.0, 1e-6, 1)
    for over_x in (False, True):
        X, R = x.to(DEV), r.to(DEV)
        tb.tern_rms_norm(0, ELEM["bf16"], T, 1, K, X, K, ELEM["bf16"], R, K, X if over_x else None, K, w.to(DEV), 0.0, 1e-6, R, K)
        close(R, y, y_bound(y, "bf16"), "y over r")
        if over_x:
            close(X, s, abs(s) * (STEP["bf16"] + 2.0 ** -23), "s over x")
