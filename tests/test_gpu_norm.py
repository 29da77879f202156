"""The norm's kernels against 64-bit references.

Bounds.  s is one fp32 addition of values that are exact in fp32 (relative 2^-24,
and the rounding of S to its type).  A thread adds at most 32 squares one after
the other, 2^-24 each, then 10 pairwise steps: the sum is within 42 * 2^-24 of
itself, its square root within half of that; the reciprocal square root and the
three products after it add 2^-22.  So y is within e = 2^-18 of itself before its
own rounding, u |y| + (fp16) 2^-25, u = 2^-8 bf16, 2^-11 fp16.  A code is the
rounding of y / a: off by 1/2 and, as |y / a| <= 127, by 127 * 2 e; a is within e.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import TYPES, UNIT, f64, randn  # noqa: E402
from gpu_util import DEV  # noqa: E402
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402

pytestmark = pytest.mark.gpu

E = 2.0 ** -18
ELEM = {"f32": tb.TERN_OUT_F32, "bf16": tb.TERN_OUT_BF16, "f16": tb.TERN_OUT_F16}
DTYPE = dict(TYPES, f32=torch.float32)
X16 = {"bf16": tb.TERN_X_BF16, "f16": tb.TERN_X_F16}
STEP = dict(UNIT, f32=2.0 ** -24)


def padded(x, pad):
    """Rows with `pad` NaN behind each, on the GPU."""
    out = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype)
    out[:, :x.shape[1]] = x
    return out.to(DEV)


def reference(x, r, w, add, eps, H):
    """(s, y) in 64 bits of [T, H * K] rows."""
    s = f64(x) if r is None else f64(x) + f64(r)
    rows = s.reshape(s.shape[0], H, -1)
    with np.errstate(all="ignore"):
        y = rows / np.sqrt((rows * rows).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
        if w is not None:
            y = y * (f64(w) + add)
    return s, y.reshape(s.shape)


def close(got, want, bound, what):
    got = f64(got)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN elsewhere"
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - want) <= bound) | (got == want)) & ~nan
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off; first {np.argwhere(bad)[0]}: {got[bad][0]} {want[bad][0]}"


def y_bound(y, t):
    return np.abs(y) * (STEP[t] + E) + (2.0 ** -25 if t == "f16" else 2.0 ** -133)


def inputs(seed, T, n, inp, res, K, t, spread=1.0):
    x = (randn(seed, T, n) * torch.exp(0.3 * randn(seed + 1, 1, n))).to(DTYPE[inp])
    r = None if res is None else (randn(seed + 2, T, n) * torch.exp(spread * randn(seed + 3, 1, n))).to(DTYPE[res])
    w = (1.0 + 0.2 * randn(seed + 4, K)).to(TYPES[t])
    return x, r, w


SIZES = [(1, 1, 8), (3, 1, 16), (5, 1, 24), (7, 1, 40), (33, 1, 64), (4, 1, 72), (9, 1, 128), (3, 1, 136), (5, 1, 256),
         (6, 1, 264), (3, 1, 512), (5, 1, 520), (17, 1, 1024), (2, 1, 1032), (3, 1, 5120), (1, 1, 8192), (2, 1, 8200),
         (2, 1, 16384), (1, 1, 16392), (2, 1, 27648), (1, 1, 32768), (3, 5, 128), (2, 40, 64), (5, 3, 80), (1, 7, 96),
         (2, 3, 1536)]


@pytest.mark.parametrize("T,H,K", SIZES)
@pytest.mark.parametrize("t,inp,res", [("bf16", "bf16", "bf16"), ("f16", "f32", "f16"), ("bf16", "f32", "f32"),
                                       ("f16", "f16", None), ("bf16", "f16", "bf16"), ("f16", "f32", None)])
def test_norm(T, H, K, t, inp, res):
    x, r, w = inputs(T * 1000 + K, T, H * K, inp, res, K, t)
    X, R = padded(x, 8), None if r is None else padded(r, 16)
    S = None if r is None else torch.full((T, H * K + 24), 7.0, dtype=DTYPE[res], device=DEV)
    Y = torch.full((T, H * K + 8), 7.0, dtype=TYPES[t], device=DEV)
    tb.tern_rms_norm(X16[t], ELEM[inp], T, H, K, X, H * K + 8, ELEM[res or "f32"], R, H * K + 16, S, H * K + 24,
                     w.to(DEV), 0.5, 1e-6, Y, H * K + 8)
    s, y = reference(x, r, w, 0.5, 1e-6, H)
    close(Y[:, :H * K], y, y_bound(y, t), "y")
    assert (Y[:, H * K:] == 7.0).all()
    if S is not None:
        close(S[:, :H * K], s, np.abs(s) * (STEP[res] + 2.0 ** -23) + 2.0 ** -25, "s")
        assert (S[:, H * K:] == 7.0).all()


@pytest.mark.parametrize("M,K", [(1, 128), (5, 256), (3, 384), (4, 1024), (3, 1152), (7, 5120), (2, 8320), (2, 27648), (1, 32768)])
@pytest.mark.parametrize("t,inp,res", [("bf16", "f32", "bf16"), ("f16", "f16", None), ("bf16", "bf16", "f32")])
def test_norm_i8(M, K, t, inp, res):
    x, r, w = inputs(M * 77 + K, M, K, inp, res, K, t)
    S = None if r is None else torch.empty((M, K), dtype=DTYPE[res], device=DEV)
    q = torch.full((M, K), 99, dtype=torch.int8, device=DEV)
    a = torch.empty((M,), device=DEV)
    tb.tern_rms_norm_i8(X16[t], ELEM[inp], M, K, x.to(DEV), K, ELEM[res or "f32"], None if r is None else r.to(DEV), K, S, K,
                        w.to(DEV), 0.0, 1e-5, q, a)
    s, y = reference(x, r, w, 0.0, 1e-5, 1)
    want_a = np.abs(y).max(1) / 127
    close(a, want_a, want_a * E, "a")
    code = f64(q).reshape(M, K // 16, 2, 8).swapaxes(2, 3).reshape(M, K)
    assert (np.abs(code - y / want_a[:, None]) <= 0.5 + 254 * E).all()
    if S is not None:
        close(S, s, np.abs(s) * (STEP[res] + 2.0 ** -23) + 2.0 ** -25, "s")


def test_codes_are_those_of_the_quantiser():
    """Codes of outputs that 16 bits hold exactly are tern_quantize_x's of those outputs, bit for bit:
    rows of +-2^-k about one size, whose norm is a power of two."""
    M, K = 5, 256
    g = torch.Generator().manual_seed(3)
    x = (2.0 * torch.randint(0, 2, (M, K), generator=g) - 1).to(torch.bfloat16)
    w = torch.exp2(torch.randint(-6, 3, (K,), generator=g).float()).to(torch.bfloat16).to(DEV)
    y = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    tb.tern_rms_norm(0, ELEM["bf16"], M, 1, K, x.to(DEV), K, 0, None, 0, None, 0, w, 0.0, 0.0, y, K)
    out = []
    for _ in range(2):
        out.append((torch.zeros(tb.tern_xq_bytes(M, K), dtype=torch.int8, device=DEV), torch.zeros(M, device=DEV)))
    tb.tern_quantize_x(y, 0, K, M, K, *out[0])
    tb.tern_rms_norm_i8(0, ELEM["bf16"], M, K, x.to(DEV), K, 0, None, 0, None, 0, w, 0.0, 0.0, *out[1])
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


@pytest.mark.parametrize("K", [128, 5120])
def test_in_place_and_without_weights(K):
    T = 6
    x, r, w = inputs(5, T, K, "bf16", "bf16", K, "bf16")
    X, R = x.to(DEV), r.to(DEV)
    tb.tern_rms_norm(0, ELEM["bf16"], T, 1, K, X, K, ELEM["bf16"], R, K, R, K, None, 123.0, 1e-6, X, K)
    s, y = reference(x, r, None, 0.0, 1e-6, 1)
    close(X, y, y_bound(y, "bf16"), "y over x")
    close(R, s, np.abs(s) * (STEP["bf16"] + 2.0 ** -23), "s over r")
    X, R, Y = x.to(DEV), r.to(DEV), torch.empty((T, K), dtype=torch.bfloat16, device=DEV)
    tb.tern_rms_norm(0, ELEM["bf16"], T, 1, K, X, K, ELEM["bf16"], R, K, X, K, w.to(DEV), 0.0, 1e-6, Y, K)
    close(X, s, np.abs(s) * (STEP["bf16"] + 2.0 ** -23), "s over x")
    assert torch.equal(R, r.to(DEV))
    # the residual's addition without its sum
    Y2 = torch.empty_like(Y)
    tb.tern_rms_norm(0, ELEM["bf16"], T, 1, K, x.to(DEV), K, ELEM["bf16"], R, K, None, 0, w.to(DEV), 0.0, 1e-6, Y2, K)
    assert torch.equal(Y, Y2)


@pytest.mark.parametrize("K", [64, 1024, 5120])
def test_sizes_of_values(K):
    """Squares beyond fp32's range on both sides, rows of zeros, one huge value, eps of none."""
    rows = [randn(1, K) * 1e25, randn(2, K) * 1e-30, torch.zeros(K), randn(3, K), torch.full((K,), 3e38), randn(4, K) * 1e-15,
            torch.full((K,), 2.0 ** -133)]
    rows[3][K // 2] = 2e30
    x = torch.stack(rows)
    for inp in ("bf16", "f32"):
        for eps in (0.0, 1e-6, 1e-30):
            v = x.to(DTYPE[inp])
            Y = torch.empty((len(rows), K), dtype=torch.bfloat16, device=DEV)
            tb.tern_rms_norm(0, ELEM[inp], len(rows), 1, K, v.to(DEV), K, 0, None, 0, None, 0, None, 0.0, eps, Y, K)
            _, y = reference(v, None, None, 0.0, eps, 1)
            close(Y, y, y_bound(y, "bf16"), f"{inp} {eps}")


@pytest.mark.parametrize("K", [128, 5120])
def test_what_is_not_finite_stays_in_its_row(K):
    x = randn(7, 4, K)
    x[1, K - 1], x[2, 0] = float("nan"), float("inf")
    v = x.to(torch.bfloat16)
    Y = torch.empty((4, K), dtype=torch.bfloat16, device=DEV)
    tb.tern_rms_norm(0, ELEM["bf16"], 4, 1, K, v.to(DEV), K, 0, None, 0, None, 0, None, 0.0, 1e-6, Y, K)
    _, y = reference(v, None, None, 0.0, 1e-6, 1)
    close(Y, y, y_bound(y, "bf16"), "y")
    q, a = torch.full((4, K), 99, dtype=torch.int8, device=DEV), torch.empty(4, device=DEV)
    tb.tern_rms_norm_i8(0, ELEM["bf16"], 4, K, v.to(DEV), K, 0, None, 0, None, 0, None, 0.0, 1e-6, q, a)
    assert torch.isnan(a).tolist() == [False, True, True, False]
    assert (q[1:3] == 0).all() and (q[0].abs().max() == 127) and (q[3].abs().max() == 127)


def test_many_rows_and_far_offsets():
    """More rows than CTAs at once; a leading dimension that puts rows 2^32 bytes and more apart."""
    T, K = 100003, 64
    x = randn(11, T, K).to(torch.bfloat16)
    Y = torch.empty((T, K), dtype=torch.bfloat16, device=DEV)
    tb.tern_rms_norm(0, ELEM["bf16"], T, 1, K, x.to(DEV), K, 0, None, 0, None, 0, None, 0.0, 1e-6, Y, K)
    _, y = reference(x, None, None, 0.0, 1e-6, 1)
    close(Y, y, y_bound(y, "bf16"), "y")
    ld = (1 << 31) + 64
    X = torch.zeros(2 * ld + 5120, dtype=torch.bfloat16, device=DEV)
    v = randn(12, 3, 5120).to(torch.bfloat16)
    for i in range(3):
        X[i * ld:i * ld + 5120] = v[i].to(DEV)
    Y = torch.empty((3, 5120), dtype=torch.bfloat16, device=DEV)
    tb.tern_rms_norm(0, ELEM["bf16"], 3, 1, 5120, X, ld, 0, None, 0, None, 0, None, 0.0, 1e-6, Y, 5120)
    _, y = reference(v, None, None, 0.0, 1e-6, 1)
    close(Y, y, y_bound(y, "bf16"), "far rows")


def test_streams_and_graphs():
    """On a stream of its own, and captured and replayed over new values."""
    T, K = 16, 5120
    x, r, w = inputs(21, T, K, "f32", "bf16", K, "bf16")
    X, R, W = x.to(DEV), r.to(DEV), w.to(DEV)
    S, Y = torch.empty_like(R), torch.empty((T, K), dtype=torch.bfloat16, device=DEV)

    def call(stream=None):
        tb.tern_rms_norm(0, ELEM["f32"], T, 1, K, X, K, ELEM["bf16"], R, K, S, K, W, 0.0, 1e-6, Y, K, stream=stream)

    call()
    want = Y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x2, r2, _ = inputs(31, T, K, "f32", "bf16", K, "bf16")
    X.copy_(x2)
    R.copy_(r2)
    graph.replay()
    _, y = reference(x2, r2, w, 0.0, 1e-6, 1)
    close(Y, y, y_bound(y, "bf16"), "replayed")


@pytest.mark.parametrize("K,lanes", [(40, 8), (64, 8), (96, 16), (128, 16), (136, 32), (256, 32)])
@pytest.mark.parametrize("t,inp,res", [("bf16", "bf16", None), ("f16", "f32", None), ("bf16", "bf16", "bf16"), ("f16", "f16", "f32"),
                                       ("bf16", "f32", "f32"), ("f16", "f32", "f16")])
def test_many_short_rows(K, lanes, t, inp, res):
    """Rows enough that a lane takes two runs of each, in 7 heads, some rows beyond fp32's squares."""
    H = 7
    T = -(-4096 * 160 // (lanes * H)) + 3
    x, r, w = inputs(K, T, H * K, inp, res, K, t)
    if inp == "f32":
        x[5::97] *= 1e25
        x[7::89] *= 1e-30
    if res in ("bf16", "f16"):                      # sums within the stream's type
        x = x.clamp(-1e4, 1e4)
    X, R = padded(x, 8), None if r is None else padded(r, 16)
    S = None if r is None else torch.full((T, H * K + 24), 7.0, dtype=DTYPE[res], device=DEV)
    Y = torch.full((T, H * K + 8), 7.0, dtype=TYPES[t], device=DEV)
    tb.tern_rms_norm(X16[t], ELEM[inp], T, H, K, X, H * K + 8, ELEM[res or "f32"], R, H * K + 16, S, H * K + 24, w.to(DEV), 0.5,
                     1e-6, Y, H * K + 8)
    s, y = reference(x, r, w, 0.5, 1e-6, H)
    close(Y[:, :H * K], y, y_bound(y, t), "y")
    assert (Y[:, H * K:] == 7.0).all()
    if r is not None:
        close(S[:, :H * K], s, np.abs(s) * (STEP[res] + 2.0 ** -23) + 2.0 ** -25, "s")


@pytest.mark.parametrize("K,lanes", [(128, 16), (256, 32)])
@pytest.mark.parametrize("inp,res", [("bf16", None), ("f32", "bf16")])
def test_codes_of_many_short_rows(K, lanes, inp, res):
    """The codes of a call with rows enough for the other form are those of its parts."""
    T = -(-4096 * 160 // lanes) + 3
    x, r, w = inputs(K + 1, T, K, inp, res, K, "bf16")
    out = []
    for parts in (1, 16):
        q, a = torch.zeros((T, K), dtype=torch.int8, device=DEV), torch.zeros(T, device=DEV)
        S = None if r is None else torch.zeros((T, K), dtype=r.dtype, device=DEV)
        for i in range(parts):
            lo, hi = T * i // parts, T * (i + 1) // parts
            X, R = x[lo:hi].to(DEV), None if r is None else r[lo:hi].to(DEV)
            tb.tern_rms_norm_i8(0, ELEM[inp], hi - lo, K, X, K, ELEM[res or "f32"], R, K, None if S is None else S[lo:hi], K,
                                w.to(DEV), 0.0, 1e-6, q[lo:hi], a[lo:hi])
        out.append((q, a, S))
    # sums of squares in another order: within 2^-18 as above, so a code moves by one at most
    assert (out[0][0].int() - out[1][0].int()).abs().max() <= 1
    assert ((out[0][1] - out[1][1]).abs() <= 2.0 ** -17 * out[1][1]).all()
    assert r is None or torch.equal(out[0][2], out[1][2])
