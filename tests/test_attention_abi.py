"""Host-side checks of the attention-side entry points (no GPU needed): bad
arguments are refused with the documented status before anything is enqueued,
and the frequency tables follow their formulas."""
import math

import numpy as np
import pytest

tbw = pytest.importorskip("ternary_bit_weight_gb300")
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402

OK, NULL, SHAPE, ALIGN, SIZE = 0, 1, 2, 3, 4
FAKE = 1 << 40       # an aligned address that is never dereferenced


def call(name, base, **change):
    args = dict(base)
    for k in change:
        assert k in args, k
    args.update(change)
    return getattr(tb.library(), name)(*args.values())


ROPE = dict(x_type=0, layout=0, T=4, D=128, rot=128, pos=FAKE, freq=FAKE, amp=1.0, Hq=8, Q=FAKE, ldq=1024, Qo=FAKE,
            ldqo=1024, Hk=2, K=FAKE, ldk=256, Ko=FAKE, ldko=256, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x_type=2), SHAPE), (dict(layout=2), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE),
    (dict(D=100), SHAPE), (dict(D=272), SHAPE), (dict(D=0), SHAPE), (dict(rot=144), SHAPE), (dict(rot=24), SHAPE),
    (dict(rot=-16), SHAPE), (dict(Hq=0), SHAPE), (dict(Hk=-1), SHAPE), (dict(ldq=1016), SHAPE), (dict(ldko=128), SHAPE),
    (dict(Q=None), NULL), (dict(Qo=None), NULL), (dict(K=None), NULL), (dict(Ko=None), NULL), (dict(pos=None), NULL),
    (dict(freq=None), NULL), (dict(Q=FAKE + 8), ALIGN), (dict(ldq=1028), ALIGN), (dict(Ko=FAKE + 2), ALIGN),
    (dict(pos=FAKE + 2), ALIGN), (dict(T=0), OK), (dict(T=0, Q=None, K=None, pos=None), OK)])
def test_rope_refusals(change, status):
    assert call("tern_rope", ROPE, **change) == status


CACHE = dict(num_pages=10, page_size=16, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE)
WRITE = dict(x_type=0, kv_type=1, T=4, Hkv=8, D=128, K=FAKE, ldk=1024, V=FAKE, ldv=1024, slots=FAKE, **CACHE, err=None,
             stream=None)
READ = dict(x_type=0, kv_type=1, T=4, Hkv=8, D=128, slots=FAKE, **CACHE, K=FAKE, ldk=1024, V=FAKE, ldv=1024, stream=None)
CACHE_REFUSALS = [
    (dict(x_type=-1), SHAPE), (dict(kv_type=3), SHAPE), (dict(kv_type=-1), SHAPE), (dict(T=-1), SHAPE),
    (dict(Hkv=0), SHAPE), (dict(D=144), SHAPE), (dict(D=8), SHAPE), (dict(page_size=0), SHAPE),
    (dict(page_size=24), SHAPE), (dict(page_size=65536), SHAPE), (dict(num_pages=-1), SHAPE), (dict(num_pages=1 << 31), SHAPE),
    (dict(ldk=1000), SHAPE), (dict(ldv=1028), ALIGN), (dict(K=None), NULL), (dict(V=None), NULL), (dict(slots=None), NULL),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(ks=None), NULL), (dict(vs=None), NULL), (dict(K=FAKE + 4), ALIGN),
    (dict(slots=FAKE + 4), ALIGN), (dict(k=FAKE + 8), ALIGN), (dict(vs=FAKE + 2), ALIGN), (dict(T=0), OK)]


@pytest.mark.parametrize("change,status", CACHE_REFUSALS)
def test_kv_refusals(change, status):
    assert call("tern_kv_write", WRITE, **change) == status
    assert call("tern_kv_read", READ, **change) == status


def test_kv_write_counter_alignment():
    assert call("tern_kv_write", WRITE, err=FAKE + 2) == ALIGN


ROPE_WRITE = dict(x_type=0, kv_type=1, layout=1, T=4, Hq=16, Hkv=8, D=128, rot=64, pos=FAKE, freq=FAKE, amp=1.0, Q=FAKE,
                  ldq=2048, Qo=FAKE, ldqo=2048, K=FAKE, ldk=1024, V=FAKE, ldv=1024, slots=FAKE, **CACHE, err=None,
                  stream=None)


@pytest.mark.parametrize("change,status", CACHE_REFUSALS + [
    (dict(layout=-1), SHAPE), (dict(rot=8), SHAPE), (dict(rot=144), SHAPE), (dict(Hq=-1), SHAPE), (dict(Q=None), NULL),
    (dict(Qo=FAKE + 2), ALIGN), (dict(ldqo=2040), SHAPE), (dict(pos=None), NULL), (dict(freq=None), NULL)])
def test_rope_kv_write_refusals(change, status):
    assert call("tern_rope_kv_write", ROPE_WRITE, **change) == status


PROMPT = dict(x_type=0, B=2, cu_q=FAKE, cu_kv=FAKE, Tq=10, Tkv=20, Hq=16, Hkv=8, D=128, causal=1, scale=0.1, Q=FAKE,
              ldq=2048, K=FAKE, ldk=1024, V=FAKE, ldv=1024, O=FAKE, ldo=2048, lse=FAKE, ws=FAKE, ws_bytes=1 << 40,
              stream=None)
PROMPT_REFUSALS = [
    (dict(x_type=2), SHAPE), (dict(B=-1), SHAPE), (dict(Tq=-1), SHAPE), (dict(Tkv=-1), SHAPE), (dict(Tq=1 << 31), SHAPE),
    (dict(Hq=12), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=136), SHAPE), (dict(D=144), SHAPE), (dict(ldq=2040), SHAPE),
    (dict(ldo=2040), SHAPE), (dict(cu_q=None), NULL), (dict(cu_kv=None), NULL), (dict(Q=None), NULL), (dict(K=None), NULL),
    (dict(V=None), NULL), (dict(O=None), NULL), (dict(cu_q=FAKE + 2), ALIGN), (dict(lse=FAKE + 2), ALIGN),
    (dict(Q=FAKE + 8), ALIGN), (dict(ldk=1028), ALIGN), (dict(O=FAKE + 8), ALIGN), (dict(B=0), OK), (dict(Tq=0), OK),
    (dict(scale=-0.1), SHAPE), (dict(scale=math.nan), SHAPE), (dict(scale=math.inf), SHAPE)]


@pytest.mark.parametrize("change,status", PROMPT_REFUSALS)
def test_prompt_refusals(change, status):
    assert call("tern_attn_prompt", PROMPT, **change) == status


DECODE = dict(x_type=0, kv_type=1, B=2, Hq=16, Hkv=8, D=128, scale=0.1, Q=FAKE, ldq=2048, **CACHE, table=FAKE, max_pages=7,
              lens=FAKE, O=FAKE, ldo=2048, lse=FAKE, ws=FAKE, ws_bytes=1 << 40, stream=None)
DECODE_REFUSALS = [
    (dict(x_type=2), SHAPE), (dict(kv_type=5), SHAPE), (dict(B=-1), SHAPE), (dict(Hq=12), SHAPE), (dict(D=160), SHAPE),
    (dict(page_size=12), SHAPE), (dict(max_pages=-1), SHAPE), (dict(max_pages=1 << 30), SHAPE), (dict(num_pages=-2), SHAPE),
    (dict(ldq=2040), SHAPE), (dict(Q=None), NULL), (dict(O=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL),
    (dict(k=None), NULL), (dict(vs=None), NULL), (dict(table=FAKE + 2), ALIGN), (dict(lens=FAKE + 1), ALIGN),
    (dict(lse=FAKE + 2), ALIGN), (dict(O=FAKE + 8), ALIGN), (dict(ldo=2052), ALIGN), (dict(B=0), OK),
    (dict(scale=-0.1), SHAPE), (dict(scale=math.nan), SHAPE)]


@pytest.mark.parametrize("change,status", DECODE_REFUSALS)
def test_decode_refusals(change, status):
    assert call("tern_attn_decode", DECODE, **change) == status


def test_workspace_bytes_are_zero_for_invalid():
    f, g = tb.tern_attn_prompt_workspace_bytes, tb.tern_attn_decode_workspace_bytes
    assert f(2, 10, 20, 16, 8, 128) > 0 and g(2, 16, 8, 128, 100) > 0
    assert f(0, 10, 20, 16, 8, 128) == f(2, 0, 20, 16, 8, 128) == f(2, 10, 20, 16, 7, 128) == f(2, 10, 20, 16, 8, 100) == 0
    assert g(0, 16, 8, 128, 100) == g(2, 16, 7, 128, 100) == g(2, 16, 8, 256, 100) == g(2, 16, 8, 128, -1) == 0


# -------------------------------------------------------------- frequencies

def test_frequencies():
    plain, amp = tb.tern_rope_freqs(128, 1e6)
    want = 1e6 ** (-2.0 * np.arange(64) / 128)
    assert amp == 1.0 and np.array_equal(np.float32(plain), want.astype(np.float32))
    linear, amp = tb.tern_rope_freqs(128, 1e6, tb.TERN_ROPE_SCALE_LINEAR, 4.0)
    assert amp == 1.0 and np.array_equal(np.float32(linear), (want / 4).astype(np.float32))
    slow, _ = tb.tern_rope_freqs(128, 1e4, tb.TERN_ROPE_SCALE_BASE, 8.0)
    base, _ = tb.tern_rope_freqs(128, 1e4)
    assert slow[0] == base[0] == 1.0
    assert abs(slow[-1] - base[-1] / 8) <= 1e-6 * base[-1]
    assert all(a <= b for a, b in zip(slow, base))


def test_frequencies_by_parts():
    trained, lo, hi, factor = 4096.0, 1.0, 32.0, 16.0
    parts, amp = tb.tern_rope_freqs(64, 1e4, tb.TERN_ROPE_SCALE_PARTS, factor, trained, lo, hi)
    f = 1e4 ** (-2.0 * np.arange(32) / 64)
    turns = trained * f / (2 * math.pi)
    keep = np.clip((turns - lo) / (hi - lo), 0, 1)
    want = (f * (keep + (1 - keep) / factor)).astype(np.float32)
    assert np.allclose(np.float32(parts), want, rtol=2.0 ** -23, atol=0)
    assert np.float32(parts[0]) == 1.0                                     # many turns: kept
    assert abs(parts[-1] - f[-1] / factor) <= 2.0 ** -22 * f[-1]           # less than one: divided
    assert abs(amp - (0.1 * math.log(factor) + 1)) <= 1e-6
    assert tb.tern_rope_freqs(64, 1e4, tb.TERN_ROPE_SCALE_PARTS, 1.0, trained)[1] == 1.0


@pytest.mark.parametrize("args", [(0, 1e4), (3, 1e4), (-2, 1e4), (258, 1e4), (64, 0.0), (64, -1.0), (64, math.inf),
                                  (64, 1e4, 9), (64, 1e4, 1, 0.0), (64, 1e4, 1, math.nan), (2, 1e4, 2, 4.0),
                                  (64, 1e4, 3, 4.0, 0.0), (64, 1e4, 3, 4.0, 10.0, 5.0, 5.0)])
def test_frequency_refusals(args):
    with pytest.raises(tb.TernError) as e:
        tb.tern_rope_freqs(*args)
    assert e.value.status == SHAPE


def test_binding_raises_with_the_status():
    with pytest.raises(tb.TernError) as e:
        tb.tern_rope(0, 0, 4, 100, 0, None, None, 1.0, 1, FAKE, 100, FAKE, 100, stream=0)
    assert e.value.status == SHAPE
    assert "TERN_ERR_SHAPE" in str(e.value)


def test_binding_converts_arguments():
    """Pointers may be None, addresses or tensors; what is neither is refused before the library is called."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(64, dtype=torch.bfloat16)

    def status(q):
        try:
            tb.tern_rope(0, 0, 4, 16, 16, FAKE, FAKE, 1.0, 1, q, 8, FAKE, 16, stream=0)   # ldq < Hq * D
        except tb.TernError as e:
            return e.status

    assert status(None) == NULL
    assert status(FAKE) == SHAPE
    assert status(x) == SHAPE
    for bad in ("x", 1.5):
        with pytest.raises((TypeError, AttributeError)):
            status(bad)
    with pytest.raises(TypeError):
        tb.tern_rope(0, 0, 4, 16, 1.5, FAKE, FAKE, 1.0, 1, FAKE, 16, FAKE, 16, stream=0)
    with pytest.raises(OverflowError):
        tb.tern_rope(1 << 40, 0, 4, 16, 16, FAKE, FAKE, 1.0, 1, FAKE, 16, FAKE, 16, stream=0)
    with pytest.raises(TypeError):
        tb.library() and tb._native.tern_rope(0, 0)
