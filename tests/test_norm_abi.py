"""Refusals of the norm's entry points (no GPU needed)."""
import math

import pytest

tbw = pytest.importorskip("ternary_bit_weight_gb300")
from test_attention_abi import ALIGN, FAKE, NULL, OK, SHAPE, call  # noqa: E402

NORM = dict(x_type=0, in_type=1, T=4, H=2, K=128, X=FAKE, ldx=256, res_type=1, R=FAKE, ldr=256, S=FAKE, lds=256, W=FAKE,
            add=0.0, eps=1e-6, Y=FAKE, ldy=256, stream=None)
NORM_I8 = dict(x_type=0, in_type=0, M=4, K=256, X=FAKE, ldx=256, res_type=0, R=FAKE, ldr=256, S=FAKE, lds=256, W=FAKE,
               add=1.0, eps=1e-6, q=FAKE, a=FAKE, stream=None)
BOTH = [
    (dict(x_type=2), SHAPE), (dict(x_type=-1), SHAPE), (dict(in_type=3), SHAPE), (dict(in_type=-1), SHAPE),
    (dict(res_type=3), SHAPE), (dict(K=0), SHAPE), (dict(K=-128), SHAPE), (dict(K=32896), SHAPE), (dict(eps=-1e-6), SHAPE),
    (dict(eps=math.nan), SHAPE), (dict(eps=math.inf), SHAPE), (dict(add=math.nan), SHAPE), (dict(add=math.inf), SHAPE),
    (dict(ldx=248), SHAPE), (dict(ldr=248), SHAPE), (dict(lds=248), SHAPE), (dict(ldx=1 << 41), SHAPE), (dict(X=None), NULL),
    (dict(R=None), NULL), (dict(X=FAKE + 8), ALIGN), (dict(R=FAKE + 2), ALIGN), (dict(S=FAKE + 4), ALIGN),
    (dict(W=FAKE + 8), ALIGN), (dict(ldx=260), ALIGN), (dict(ldr=257), ALIGN), (dict(lds=260), ALIGN)]


@pytest.mark.parametrize("change,status", BOTH + [
    (dict(T=-1), SHAPE), (dict(T=(1 << 30) + 1), SHAPE), (dict(T=1 << 20, H=4096, ldx=1 << 20), SHAPE), (dict(H=0), SHAPE),
    (dict(H=4097), SHAPE), (dict(K=132), SHAPE), (dict(K=4), SHAPE), (dict(Y=None), NULL), (dict(ldy=248), SHAPE),
    (dict(ldy=260), ALIGN), (dict(Y=FAKE + 8), ALIGN), (dict(T=0), OK), (dict(T=0, X=None, Y=None), OK)])
def test_norm_refusals(change, status):
    assert call("tern_rms_norm", NORM, **change) == status


@pytest.mark.parametrize("change,status", BOTH + [
    (dict(M=-1), SHAPE), (dict(K=136), SHAPE), (dict(K=64), SHAPE), (dict(q=None), NULL), (dict(a=None), NULL),
    (dict(q=FAKE + 8), ALIGN), (dict(a=FAKE + 2), ALIGN), (dict(M=0), OK)])
def test_norm_i8_refusals(change, status):
    assert call("tern_rms_norm_i8", NORM_I8, **change) == status


APART = dict(S=FAKE + 4096, Y=FAKE + 8192, R=FAKE + 12288)


@pytest.mark.parametrize("change", [
    dict(Y=FAKE + 4096),                               # both outputs in one place
    dict(Y=FAKE, ldy=264), dict(Y=FAKE, in_type=0), dict(Y=FAKE, in_type=2), dict(Y=FAKE, x_type=1),
    dict(S=FAKE, lds=264), dict(S=FAKE, res_type=2), dict(S=FAKE, res_type=0), dict(S=FAKE + 12288, lds=264)])
def test_in_place_only_element_by_element(change):
    """An output in its input's place, by another type or leading dimension, would be read after it is written."""
    assert call("tern_rms_norm", NORM, **{**APART, **change}) == SHAPE


@pytest.mark.parametrize("change", [dict(S=FAKE, lds=264), dict(S=FAKE, res_type=1), dict(S=FAKE + 12288, lds=264)])
def test_i8_in_place_only_element_by_element(change):
    assert call("tern_rms_norm_i8", NORM_I8, **{**dict(S=FAKE + 4096, R=FAKE + 12288), **change}) == SHAPE


@pytest.mark.parametrize("change", [
    dict(Y=FAKE + 12288, res_type=0), dict(Y=FAKE + 12288, res_type=2), dict(Y=FAKE + 12288, ldy=264),
    dict(Y=FAKE + 12288, S=None, res_type=0), dict(Y=FAKE + 12288, S=None, x_type=1), dict(Y=FAKE + 16384, W=FAKE + 16384),
    dict(S=FAKE + 16384, W=FAKE + 16384)])
def test_outputs_over_the_stream_and_the_weights(change):
    """The normalised rows in the residual stream's place by another type or leading dimension, an output in the weights'."""
    assert call("tern_rms_norm", NORM, **{**APART, **change}) == SHAPE


I8_APART = dict(X=FAKE, R=FAKE + 4096, S=FAKE + 8192, W=FAKE + 12288, q=FAKE + 16384, a=FAKE + 20480)


@pytest.mark.parametrize("out", ["q", "a"])
@pytest.mark.parametrize("over", ["X", "R", "S", "W"])
def test_codes_and_factors_have_a_place_of_their_own(out, over):
    assert call("tern_rms_norm_i8", NORM_I8, **{**I8_APART, out: I8_APART[over]}) == SHAPE
    if over != "W":
        assert call("tern_rms_norm_i8", NORM_I8, **{**I8_APART, "R": I8_APART["S"], out: I8_APART["S"]}) == SHAPE


def test_codes_beside_their_factors():
    assert call("tern_rms_norm_i8", NORM_I8, **{**I8_APART, "a": I8_APART["q"]}) == SHAPE


@pytest.mark.parametrize("change,status", [(dict(H=4096, T=4, K=8, ldx=32768, ldr=32768, lds=32768, ldy=32768, W=FAKE + 8), ALIGN),
                                           (dict(ldy=(1 << 40) + 8), SHAPE), (dict(ldr=(1 << 40) + 8), SHAPE)])
def test_limits(change, status):
    """The largest head count passes the shape (the weights' alignment is what is refused), leading dimensions end at 2^40."""
    assert call("tern_rms_norm", NORM, **{**APART, **change}) == status
