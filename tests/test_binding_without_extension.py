"""The binding where the extension module was not built for the interpreter: importing it
and the linear layer's calls need no extension, and the attention-side calls go
through ctypes with the same conversions and refusals."""
import subprocess
import sys

import pytest

pytest.importorskip("ternary_bit_weight_gb300")
from conftest import ROOT  # noqa: E402
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402
from ternary_bit_weight_gb300 import build  # noqa: E402

FAKE = 1 << 40       # an aligned address that is never dereferenced
NULL, SHAPE = 1, 2

IMPORT = """
import os, sys
sys.path.insert(0, {root!r})
exists = os.path.exists
os.path.exists = lambda p: "_tern_python" not in str(p) and exists(p)
from ternary_bit_weight_gb300 import binding as tb
print(tb.tern_workspace_bytes(4, 64, 256) > 0, tb.tern_attn_decode_workspace_bytes(1, 8, 2, 128, 100) > 0)
try:
    tb.tern_rope(0, 0, 4, 16, 16, {fake}, {fake}, 1.0, 1, {fake}, 8, {fake}, 16, stream=0)
except tb.TernError as e:
    print(e.status)
"""


def test_import_without_the_extension():
    run = subprocess.run([sys.executable, "-c", IMPORT.format(root=ROOT, fake=FAKE)], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    assert run.stdout.split() == ["True", "True", str(SHAPE)]


def test_extension_is_built_for_this_interpreter():
    """Another interpreter does not find it, and builds its own."""
    import sysconfig
    assert build.PY_LIB.endswith("_tern_python" + sysconfig.get_config_var("EXT_SUFFIX"))
    assert (build.python_headers() is None) == isinstance(tb._native, tb._CtypesCalls)


@pytest.fixture
def through_ctypes(monkeypatch):
    monkeypatch.setattr(tb, "_native", tb._CtypesCalls())


def test_conversions_through_ctypes(through_ctypes):
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
        tb._native.tern_rope(0, 0)


@pytest.mark.parametrize("name", ["tern_rope", "tern_kv_write", "tern_rope_kv_write", "tern_kv_read", "tern_attn_prompt",
                                  "tern_attn_decode"])
def test_both_ways_answer_alike(name):
    """All arguments zero: the same status from both, so the same arguments in the same places."""
    n = len(getattr(tb.library(), name).argtypes)
    ways = [tb._native, tb._CtypesCalls()]
    kinds = getattr(tb.library(), name).argtypes
    import ctypes
    zero = [0.5 if k is ctypes.c_float else None if k is ctypes.c_void_p else 0 for k in kinds]
    want = getattr(ways[1], name)(*zero)
    assert getattr(ways[0], name)(*zero) == want
    for i, k in enumerate(kinds):     # one argument at a time
        if k is ctypes.c_void_p:
            continue
        some = list(zero)
        some[i] = 16
        assert getattr(ways[0], name)(*some) == getattr(ways[1], name)(*some)
    for way in ways:
        with pytest.raises(TypeError):
            getattr(way, name)(*zero[:n - 1])
