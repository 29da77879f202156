"""ctypes binding of libtern's C ABI (include/tern.h).

Argument marshalling only: every step of the layer runs in libtern's CUDA
kernels.  Functions carry the C names; tensor arguments may be torch
tensors (their ``data_ptr()`` is passed) or raw integer addresses, and
``stream`` may be a ``torch.cuda.Stream``, a raw ``cudaStream_t`` integer or
None (the current torch stream).  A non-zero status raises ``TernError``.
If the library has not been built, importing this module raises.

The attention-side calls and the norms go through a small extension module
(csrc/tern_python.c) instead of ctypes, which converts their many arguments
three times as fast; where it was not built for this interpreter (no Python
headers), they go through ctypes to the same library.  The functions below are
the same to a caller.
"""
from __future__ import annotations

import ctypes
import importlib.util
import operator
import os

from . import build as _build

TERN_OK = 0
TERN_X_BF16, TERN_X_F16 = 0, 1
TERN_OUT_F32, TERN_OUT_BF16, TERN_OUT_F16 = 0, 1, 2
TERN_ROPE_HALF, TERN_ROPE_INTERLEAVED = 0, 1
TERN_ROPE_SCALE_NONE, TERN_ROPE_SCALE_LINEAR, TERN_ROPE_SCALE_BASE, TERN_ROPE_SCALE_PARTS = 0, 1, 2, 3
TERN_KV_X16, TERN_KV_E4M3, TERN_KV_I8 = 0, 1, 2
STATUS_NAMES = {0: "TERN_OK", 1: "TERN_ERR_NULL", 2: "TERN_ERR_SHAPE", 3: "TERN_ERR_ALIGN",
                4: "TERN_ERR_SIZE", 5: "TERN_ERR_UNSUPPORTED", 6: "TERN_ERR_CUDA"}

# Every symbol include/tern.h declares.
EXPORTED = ("tern_status_string", "tern_version", "tern_pack", "tern_unpack", "tern_tiled_bytes",
            "tern_repack", "tern_unrepack", "tern_workspace_bytes", "tern_linear",
            "tern_linear_multi", "tern_linear_noalloc", "tern_linear_ex", "tern_tiled_glu_bytes",
            "tern_repack_glu", "tern_swiglu_workspace_bytes", "tern_linear_swiglu",
            "tern_workspace_error", "tern_workspace_reset", "tern_xq_bytes", "tern_quantize_x",
            "tern_i8_workspace_bytes", "tern_linear_i8", "tern_tiled_s8_bytes", "tern_quantize_scales",
            "tern_repack_s8", "tern_linear_s8", "tern_unit_count", "tern_zero_units", "tern_linear_sparse",
            "tern_grouped_workspace_bytes", "tern_linear_grouped", "tern_repack_grouped",
            "tern_rope_freqs", "tern_rope", "tern_kv_write", "tern_rope_kv_write", "tern_kv_read",
            "tern_attn_prompt_workspace_bytes", "tern_attn_prompt", "tern_attn_decode_workspace_bytes",
            "tern_attn_decode", "tern_rms_norm", "tern_rms_norm_i8", "tern_attn_weights", "tern_kv_keep",
            "tern_kv_compact")

MAX_GROUP = 8


class TernError(RuntimeError):
    def __init__(self, status: int, func: str):
        self.status = status
        super().__init__(f"{func}: {status_string(status)}")


def _load():
    if not os.path.exists(_build.LIB):
        raise ImportError(f"libtern.so is not built ({_build.LIB}); run "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(_build.LIB)
    i64, vp, sz, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    lib.tern_status_string.argtypes = [i32]
    lib.tern_status_string.restype = ctypes.c_char_p
    lib.tern_version.argtypes = []
    lib.tern_version.restype = i32
    lib.tern_pack.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.tern_pack.restype = i32
    lib.tern_unpack.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.tern_unpack.restype = i32
    lib.tern_tiled_bytes.argtypes = [i64, i64]
    lib.tern_tiled_bytes.restype = sz
    lib.tern_repack.argtypes = [vp, vp, i64, i64, vp, sz, vp, vp]
    lib.tern_repack.restype = i32
    lib.tern_unrepack.argtypes = [vp, i64, i64, vp, vp, vp, vp]
    lib.tern_unrepack.restype = i32
    lib.tern_workspace_bytes.argtypes = [i64, i64, i64]
    lib.tern_workspace_bytes.restype = sz
    lib.tern_linear.argtypes = [vp, i64, vp, i64, i64, i64, vp, i64, vp, sz, vp]
    lib.tern_linear.restype = i32
    lib.tern_linear_multi.argtypes = [vp, i64, vp, i64, i64, i32, ctypes.POINTER(i64),
                                      ctypes.POINTER(vp), ctypes.POINTER(i64), vp, sz, vp]
    lib.tern_linear_multi.restype = i32
    lib.tern_linear_noalloc.argtypes = [vp, i64, vp, i64, i64, i64, vp, i64, vp]
    lib.tern_linear_noalloc.restype = i32
    lib.tern_linear_ex.argtypes = [vp, i32, i64, vp, i64, i64, i32, ctypes.POINTER(i64),
                                   ctypes.POINTER(vp), ctypes.POINTER(i64), i32, vp, sz, vp]
    lib.tern_linear_ex.restype = i32
    lib.tern_grouped_workspace_bytes.argtypes = [i64, i32, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    lib.tern_grouped_workspace_bytes.restype = sz
    lib.tern_linear_grouped.argtypes = [i32, i64, i32, ctypes.POINTER(vp), ctypes.POINTER(i64), ctypes.POINTER(vp),
                                        ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(vp),
                                        ctypes.POINTER(i64), i32, vp, sz, vp]
    lib.tern_linear_grouped.restype = i32
    lib.tern_repack_grouped.argtypes = [i32, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(i64),
                                        ctypes.POINTER(i64), ctypes.POINTER(vp), ctypes.POINTER(sz), vp, vp]
    lib.tern_repack_grouped.restype = i32
    lib.tern_tiled_glu_bytes.argtypes = [i64, i64]
    lib.tern_tiled_glu_bytes.restype = sz
    lib.tern_repack_glu.argtypes = [vp, vp, vp, vp, i64, i64, vp, sz, vp, vp]
    lib.tern_repack_glu.restype = i32
    lib.tern_swiglu_workspace_bytes.argtypes = [i64, i64, i64]
    lib.tern_swiglu_workspace_bytes.restype = sz
    lib.tern_linear_swiglu.argtypes = [vp, i32, i64, vp, i64, i64, i64, vp, i64, i32, vp, sz, vp]
    lib.tern_linear_swiglu.restype = i32
    lib.tern_workspace_error.argtypes = [vp, vp, vp]
    lib.tern_workspace_error.restype = i32
    lib.tern_workspace_reset.argtypes = [vp, sz, vp]
    lib.tern_workspace_reset.restype = i32
    lib.tern_xq_bytes.argtypes = [i64, i64]
    lib.tern_xq_bytes.restype = sz
    lib.tern_quantize_x.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp]
    lib.tern_quantize_x.restype = i32
    lib.tern_i8_workspace_bytes.argtypes = [i64, i64, i64]
    lib.tern_i8_workspace_bytes.restype = sz
    lib.tern_linear_i8.argtypes = [vp, vp, vp, i64, i64, i64, vp, i64, i32, vp, sz, vp]
    lib.tern_linear_i8.restype = i32
    lib.tern_tiled_s8_bytes.argtypes = [i64, i64]
    lib.tern_tiled_s8_bytes.restype = sz
    lib.tern_quantize_scales.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.tern_quantize_scales.restype = i32
    lib.tern_repack_s8.argtypes = [vp, vp, vp, i64, i64, vp, sz, vp, vp]
    lib.tern_repack_s8.restype = i32
    lib.tern_linear_s8.argtypes = list(lib.tern_linear_ex.argtypes)
    lib.tern_linear_s8.restype = i32
    lib.tern_unit_count.argtypes = [i64, i64]
    lib.tern_unit_count.restype = sz
    lib.tern_zero_units.argtypes = [vp, i64, i64, vp, vp]
    lib.tern_zero_units.restype = i32
    lib.tern_linear_sparse.argtypes = [vp, i32, i64, vp, vp, i64, i64, i32, ctypes.POINTER(i64),
                                       ctypes.POINTER(vp), ctypes.POINTER(i64), i32, vp, sz, vp]
    lib.tern_linear_sparse.restype = i32
    f32, f64 = ctypes.c_float, ctypes.c_double
    lib.tern_rope_freqs.argtypes = [i64, f64, i32, f64, f64, f64, f64, vp, vp]
    lib.tern_rope_freqs.restype = i32
    lib.tern_rope.argtypes = [i32, i32, i64, i64, i64, vp, vp, f32, i64, vp, i64, vp, i64, i64, vp, i64, vp, i64, vp]
    lib.tern_rope.restype = i32
    cache = [i64, i64, vp, vp, vp, vp]
    lib.tern_kv_write.argtypes = [i32, i32, i64, i64, i64, vp, i64, vp, i64, vp, *cache, vp, vp]
    lib.tern_kv_write.restype = i32
    lib.tern_rope_kv_write.argtypes = [i32, i32, i32, i64, i64, i64, i64, i64, vp, vp, f32, vp, i64, vp, i64, vp, i64,
                                       vp, i64, vp, *cache, vp, vp]
    lib.tern_rope_kv_write.restype = i32
    lib.tern_kv_read.argtypes = [i32, i32, i64, i64, i64, vp, *cache, vp, i64, vp, i64, vp]
    lib.tern_kv_read.restype = i32
    lib.tern_attn_prompt_workspace_bytes.argtypes = [i64] * 6
    lib.tern_attn_prompt_workspace_bytes.restype = sz
    lib.tern_attn_prompt.argtypes = [i32, i64, vp, vp, i64, i64, i64, i64, i64, i32, f32, vp, i64, vp, i64, vp, i64,
                                     vp, i64, vp, vp, sz, vp]
    lib.tern_attn_prompt.restype = i32
    lib.tern_attn_decode_workspace_bytes.argtypes = [i64] * 5
    lib.tern_attn_decode_workspace_bytes.restype = sz
    lib.tern_attn_decode.argtypes = [i32, i32, i64, i64, i64, i64, f32, vp, i64, *cache, vp, i64, vp, vp, i64, vp, vp,
                                     sz, vp]
    lib.tern_attn_decode.restype = i32
    lib.tern_attn_weights.argtypes = [i32, i32, i64, vp, i64, i64, i64, i64, f32, vp, i64, vp, i64, i64, vp, vp, vp, i64, vp,
                                      vp, f32, vp, vp, vp]
    lib.tern_attn_weights.restype = i32
    lib.tern_kv_keep.argtypes = [i64, i64, i64, i64, vp, vp, i64, vp, i64, i64, i64, vp, vp, vp]
    lib.tern_kv_keep.restype = i32
    lib.tern_kv_compact.argtypes = [i32, i64, i64, i64, *cache, vp, vp, i64, vp, i64, vp, i64, vp, vp]
    lib.tern_kv_compact.restype = i32
    norm = [vp, i64, i32, vp, i64, vp, i64, vp, f32, f32]
    lib.tern_rms_norm.argtypes = [i32, i32, i64, i64, i64, *norm, vp, i64, vp]
    lib.tern_rms_norm.restype = i32
    lib.tern_rms_norm_i8.argtypes = [i32, i32, i64, i64, *norm, vp, vp, vp]
    lib.tern_rms_norm_i8.restype = i32
    return lib


_lib = _load()


class _CtypesCalls:
    """The extension module's calls through ctypes, with its conversions and refusals."""

    def __getattr__(self, name):
        fn = getattr(_lib, name)
        kinds = fn.argtypes

        def pointer(x):
            if x is None or isinstance(x, int):
                return x
            return x.data_ptr()

        def integer(bits):
            def convert(x):
                x = operator.index(x)
                if not -(1 << (bits - 1)) <= x < 1 << (bits - 1):
                    raise OverflowError(f"argument does not fit {bits} bits")
                return x
            return convert

        convert = {ctypes.c_void_p: pointer, ctypes.c_int: integer(32), ctypes.c_int64: integer(64),
                   ctypes.c_size_t: integer(64), ctypes.c_float: float}
        convert = [convert[k] for k in kinds]

        def call(*args):
            if len(args) != len(convert):
                raise TypeError(f"expected {len(convert)} arguments, got {len(args)}")
            return fn(*[c(x) for c, x in zip(convert, args)])

        setattr(self, name, call)
        return call


def _load_native():
    if not os.path.exists(_build.PY_LIB):
        return _CtypesCalls()
    spec = importlib.util.spec_from_file_location("_tern_python", _build.PY_LIB)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


_native = _load_native()


def library():
    """The loaded ctypes library object."""
    return _lib


def library_path() -> str:
    return _build.LIB


def _p(x):
    """Device/host address of a tensor or an int (None -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None


def _current_stream():
    """cudaStream_t of torch's current stream.  Through torch's raw-stream
    lookup, 0.1 us: building a ``torch.cuda.Stream`` object takes 3 us, a third
    of a small call's time on the host."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        torch.cuda.init()
        get, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        _raw_stream = lambda: get(device())  # noqa: E731
    return _raw_stream()


def _s(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, func: str):
    if status != TERN_OK:
        raise TernError(status, func)


def status_string(status: int) -> str:
    return _lib.tern_status_string(status).decode()


def tern_status_string(status: int) -> str:
    return status_string(status)


def tern_version() -> int:
    return int(_lib.tern_version())


def tern_pack(t, N: int, K: int, packed, err=None, stream=None):
    _check(_lib.tern_pack(_p(t), N, K, _p(packed), _p(err), _s(stream)), "tern_pack")


def tern_unpack(packed, N: int, K: int, t, err=None, stream=None):
    _check(_lib.tern_unpack(_p(packed), N, K, _p(t), _p(err), _s(stream)), "tern_unpack")


def tern_tiled_bytes(N: int, K: int) -> int:
    return int(_lib.tern_tiled_bytes(N, K))


def tern_repack(packed, scales, N: int, K: int, tiled, tiled_bytes: int | None = None, err=None,
                stream=None):
    if tiled_bytes is None:
        tiled_bytes = tiled.numel() * tiled.element_size()
    _check(_lib.tern_repack(_p(packed), _p(scales), N, K, _p(tiled), tiled_bytes, _p(err), _s(stream)),
           "tern_repack")


def tern_unrepack(tiled, N: int, K: int, packed, scales, err=None, stream=None):
    _check(_lib.tern_unrepack(_p(tiled), N, K, _p(packed), _p(scales), _p(err), _s(stream)),
           "tern_unrepack")


def tern_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.tern_workspace_bytes(M, N, K))


def tern_linear(X, ldx: int, tiled, M: int, N: int, K: int, Y, ldy: int, ws=None,
                ws_bytes: int | None = None, stream=None):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None or isinstance(ws, int) else ws.numel() * ws.element_size()
    _check(_lib.tern_linear(_p(X), ldx, _p(tiled), M, N, K, _p(Y), ldy, _p(ws), ws_bytes, _s(stream)),
           "tern_linear")


def tern_linear_multi(X, ldx: int, tiled, M: int, K: int, n_sizes, Ys, ldys, ws=None,
                      ws_bytes: int | None = None, stream=None):
    n_out = len(n_sizes)
    sizes = (ctypes.c_int64 * n_out)(*[int(v) for v in n_sizes])
    ptrs = (ctypes.c_void_p * n_out)(*[_p(y) for y in Ys])
    lds = (ctypes.c_int64 * n_out)(*[int(v) for v in ldys])
    if ws_bytes is None:
        ws_bytes = 0 if ws is None or isinstance(ws, int) else ws.numel() * ws.element_size()
    _check(_lib.tern_linear_multi(_p(X), ldx, _p(tiled), M, K, n_out, sizes, ptrs, lds, _p(ws),
                                  ws_bytes, _s(stream)), "tern_linear_multi")


def tern_linear_noalloc(X, ldx: int, tiled, M: int, N: int, K: int, Y, ldy: int, stream=None):
    """tern_linear with the library's built-in scratch instead of a workspace."""
    _check(_lib.tern_linear_noalloc(_p(X), ldx, _p(tiled), M, N, K, _p(Y), ldy, _s(stream)),
           "tern_linear_noalloc")


def _nbytes(t):
    return 0 if t is None or isinstance(t, int) else t.numel() * t.element_size()


def tern_linear_ex(X, x_type: int, ldx: int, tiled, M: int, K: int, n_sizes, Ys, ldys, out_type: int,
                   ws=None, ws_bytes: int | None = None, stream=None):
    """Multi-output linear with the activation and output element types chosen."""
    n_out = len(n_sizes)
    sizes = (ctypes.c_int64 * n_out)(*[int(v) for v in n_sizes])
    ptrs = (ctypes.c_void_p * n_out)(*[_p(y) for y in Ys])
    lds = (ctypes.c_int64 * n_out)(*[int(v) for v in ldys])
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    _check(_lib.tern_linear_ex(_p(X), x_type, ldx, _p(tiled), M, K, n_out, sizes, ptrs, lds, out_type,
                               _p(ws), ws_bytes, _s(stream)), "tern_linear_ex")


def _i64s(vals):
    return (ctypes.c_int64 * len(vals))(*[int(v) for v in vals])


def _ptrs(vals):
    return (ctypes.c_void_p * len(vals))(*[_p(v) for v in vals])


def tern_grouped_workspace_bytes(M: int, Ns, Ks) -> int:
    return int(_lib.tern_grouped_workspace_bytes(M, len(Ns), _i64s(Ns), _i64s(Ks)))


def tern_linear_grouped(x_type: int, M: int, Xs, ldxs, tiled, Ns, Ks, Ys, ldys, out_type: int, ws=None,
                        ws_bytes: int | None = None, stream=None):
    """Independent linears (one output each, the same M) in one launch: the
    streaming kernel for M <= 16, the tensor-core GEMM above."""
    count = len(Ns)
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    _check(_lib.tern_linear_grouped(x_type, M, count, _ptrs(Xs), _i64s(ldxs), _ptrs(tiled), _i64s(Ns), _i64s(Ks),
                                    _ptrs(Ys), _i64s(ldys), out_type, _p(ws), ws_bytes, _s(stream)),
           "tern_linear_grouped")


def tern_repack_grouped(packed, scales, Ns, Ks, tiled, tiled_bytes=None, err=None, stream=None):
    """Several disk -> tiled repacks in one launch."""
    count = len(Ns)
    if tiled_bytes is None:
        tiled_bytes = [_nbytes(t) for t in tiled]
    sizes = (ctypes.c_size_t * count)(*[int(v) for v in tiled_bytes])
    _check(_lib.tern_repack_grouped(count, _ptrs(packed), _ptrs(scales), _i64s(Ns), _i64s(Ks), _ptrs(tiled), sizes,
                                    _p(err), _s(stream)), "tern_repack_grouped")


def tern_tiled_glu_bytes(I: int, K: int) -> int:
    return int(_lib.tern_tiled_glu_bytes(I, K))


def tern_repack_glu(packed_gate, scales_gate, packed_up, scales_up, I: int, K: int, tiled,
                    tiled_bytes: int | None = None, err=None, stream=None):
    if tiled_bytes is None:
        tiled_bytes = _nbytes(tiled)
    _check(_lib.tern_repack_glu(_p(packed_gate), _p(scales_gate), _p(packed_up), _p(scales_up), I, K,
                                _p(tiled), tiled_bytes, _p(err), _s(stream)), "tern_repack_glu")


def tern_swiglu_workspace_bytes(M: int, I: int, K: int) -> int:
    return int(_lib.tern_swiglu_workspace_bytes(M, I, K))


def tern_linear_swiglu(X, x_type: int, ldx: int, tiled_glu, M: int, I: int, K: int, H, ldh: int,
                       out_type: int, ws=None, ws_bytes: int | None = None, stream=None):
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    _check(_lib.tern_linear_swiglu(_p(X), x_type, ldx, _p(tiled_glu), M, I, K, _p(H), ldh, out_type,
                                   _p(ws), ws_bytes, _s(stream)), "tern_linear_swiglu")


def tern_workspace_error(ws, stream=None) -> int:
    """The workspace's error word (waits for ``stream`` to reach this point)."""
    out = ctypes.c_int32(0)
    _check(_lib.tern_workspace_error(_p(ws), ctypes.addressof(out), _s(stream)), "tern_workspace_error")
    return int(out.value)


def tern_workspace_reset(ws, ws_bytes: int | None = None, stream=None):
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    _check(_lib.tern_workspace_reset(_p(ws), ws_bytes, _s(stream)), "tern_workspace_reset")


def tern_xq_bytes(M: int, K: int) -> int:
    return int(_lib.tern_xq_bytes(M, K))


def tern_quantize_x(X, x_type: int, ldx: int, M: int, K: int, xq, a, stream=None):
    _check(_lib.tern_quantize_x(_p(X), x_type, ldx, M, K, _p(xq), _p(a), _s(stream)), "tern_quantize_x")


def tern_i8_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.tern_i8_workspace_bytes(M, N, K))


def tern_linear_i8(xq, a, tiled, M: int, N: int, K: int, Y, ldy: int, out_type: int = 0, ws=None,
                   ws_bytes: int | None = None, stream=None):
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    _check(_lib.tern_linear_i8(_p(xq), _p(a), _p(tiled), M, N, K, _p(Y), ldy, out_type, _p(ws), ws_bytes,
                               _s(stream)), "tern_linear_i8")


def tern_tiled_s8_bytes(N: int, K: int) -> int:
    return int(_lib.tern_tiled_s8_bytes(N, K))


def tern_quantize_scales(scales, N: int, K: int, q8, f, stream=None):
    _check(_lib.tern_quantize_scales(_p(scales), N, K, _p(q8), _p(f), _s(stream)), "tern_quantize_scales")


def tern_repack_s8(packed, q8, f, N: int, K: int, tiled, tiled_bytes: int | None = None, err=None, stream=None):
    if tiled_bytes is None:
        tiled_bytes = _nbytes(tiled)
    _check(_lib.tern_repack_s8(_p(packed), _p(q8), _p(f), N, K, _p(tiled), tiled_bytes, _p(err), _s(stream)),
           "tern_repack_s8")


def tern_linear_s8(X, x_type: int, ldx: int, tiled_s8, M: int, K: int, n_sizes, Ys, ldys, out_type: int,
                   ws=None, ws_bytes: int | None = None, stream=None):
    n_out = len(n_sizes)
    sizes = (ctypes.c_int64 * n_out)(*[int(v) for v in n_sizes])
    ptrs = (ctypes.c_void_p * n_out)(*[_p(y) for y in Ys])
    lds = (ctypes.c_int64 * n_out)(*[int(v) for v in ldys])
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    _check(_lib.tern_linear_s8(_p(X), x_type, ldx, _p(tiled_s8), M, K, n_out, sizes, ptrs, lds, out_type,
                               _p(ws), ws_bytes, _s(stream)), "tern_linear_s8")


def tern_unit_count(N: int, K: int) -> int:
    return int(_lib.tern_unit_count(N, K))


def tern_zero_units(tiled, N: int, K: int, flags, stream=None):
    _check(_lib.tern_zero_units(_p(tiled), N, K, _p(flags), _s(stream)), "tern_zero_units")


def tern_linear_sparse(X, x_type: int, ldx: int, tiled, flags, M: int, K: int, n_sizes, Ys, ldys, out_type: int,
                       ws=None, ws_bytes: int | None = None, stream=None):
    n_out = len(n_sizes)
    sizes = (ctypes.c_int64 * n_out)(*[int(v) for v in n_sizes])
    ptrs = (ctypes.c_void_p * n_out)(*[_p(y) for y in Ys])
    lds = (ctypes.c_int64 * n_out)(*[int(v) for v in ldys])
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    _check(_lib.tern_linear_sparse(_p(X), x_type, ldx, _p(tiled), _p(flags), M, K, n_out, sizes, ptrs, lds,
                                   out_type, _p(ws), ws_bytes, _s(stream)), "tern_linear_sparse")


def tern_rope_freqs(rot_dim: int, base: float, scaling: int = TERN_ROPE_SCALE_NONE, factor: float = 1.0,
                    trained_len: float = 1.0, turns_low: float = 1.0, turns_high: float = 32.0):
    """Frequencies of rotary positions: (list of rot_dim/2 fp32 values, amplitude)."""
    freq = (ctypes.c_float * max(1, int(rot_dim) // 2))()
    amplitude = ctypes.c_float(0.0)
    _check(_lib.tern_rope_freqs(rot_dim, base, scaling, factor, trained_len, turns_low, turns_high,
                                ctypes.addressof(freq), ctypes.addressof(amplitude)), "tern_rope_freqs")
    return list(freq), float(amplitude.value)


def tern_rope(x_type: int, layout: int, T: int, D: int, rot_dim: int, pos, inv_freq, amplitude: float, Hq: int, Q,
              ldq: int, Qo, ldqo: int, Hk: int = 0, K=None, ldk: int = 0, Ko=None, ldko: int = 0, stream=None):
    """Rotary positions of queries and (Hk > 0) keys in one pass."""
    _check(_native.tern_rope(x_type, layout, T, D, rot_dim, pos, inv_freq, amplitude, Hq, Q, ldq, Qo, ldqo,
                             Hk, K, ldk, Ko, ldko, _s(stream)), "tern_rope")


def tern_kv_write(x_type: int, kv_type: int, T: int, Hkv: int, D: int, K, ldk: int, V, ldv: int, slots, num_pages: int,
                  page_size: int, kcache, vcache, kscale=None, vscale=None, err=None, stream=None):
    """Store T tokens' keys and values in the paged cache."""
    _check(_native.tern_kv_write(x_type, kv_type, T, Hkv, D, K, ldk, V, ldv, slots, num_pages, page_size,
                                 kcache, vcache, kscale, vscale, err, _s(stream)), "tern_kv_write")


def tern_rope_kv_write(x_type: int, kv_type: int, layout: int, T: int, Hq: int, Hkv: int, D: int, rot_dim: int, pos,
                       inv_freq, amplitude: float, Q, ldq: int, Qo, ldqo: int, K, ldk: int, V, ldv: int, slots,
                       num_pages: int, page_size: int, kcache, vcache, kscale=None, vscale=None, err=None, stream=None):
    """tern_rope of queries and keys and tern_kv_write of the rotated keys in one pass."""
    _check(_native.tern_rope_kv_write(x_type, kv_type, layout, T, Hq, Hkv, D, rot_dim, pos, inv_freq, amplitude,
                                      Q, ldq, Qo, ldqo, K, ldk, V, ldv, slots, num_pages, page_size,
                                      kcache, vcache, kscale, vscale, err, _s(stream)),
           "tern_rope_kv_write")


def tern_kv_read(x_type: int, kv_type: int, T: int, Hkv: int, D: int, slots, num_pages: int, page_size: int, kcache,
                 vcache, kscale, vscale, K, ldk: int, V, ldv: int, stream=None):
    """Read T tokens of the paged cache back as rows of keys and values."""
    _check(_native.tern_kv_read(x_type, kv_type, T, Hkv, D, slots, num_pages, page_size, kcache, vcache,
                                kscale, vscale, K, ldk, V, ldv, _s(stream)), "tern_kv_read")


def tern_attn_prompt_workspace_bytes(B: int, Tq: int, Tkv: int, Hq: int, Hkv: int, D: int) -> int:
    return int(_lib.tern_attn_prompt_workspace_bytes(B, Tq, Tkv, Hq, Hkv, D))


def tern_attn_prompt(x_type: int, B: int, cu_q, cu_kv, Tq: int, Tkv: int, Hq: int, Hkv: int, D: int, causal: bool,
                     scale: float, Q, ldq: int, K, ldk: int, V, ldv: int, O, ldo: int, lse=None, ws=None,
                     ws_bytes: int | None = None, stream=None):
    """Attention over B packed prompts."""
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    _check(_native.tern_attn_prompt(x_type, B, cu_q, cu_kv, Tq, Tkv, Hq, Hkv, D, causal, scale, Q, ldq,
                                    K, ldk, V, ldv, O, ldo, lse, ws, ws_bytes, _s(stream)),
           "tern_attn_prompt")


def tern_attn_decode_workspace_bytes(B: int, Hq: int, Hkv: int, D: int, max_len: int) -> int:
    return int(_lib.tern_attn_decode_workspace_bytes(B, Hq, Hkv, D, max_len))


def tern_attn_decode(x_type: int, kv_type: int, B: int, Hq: int, Hkv: int, D: int, scale: float, Q, ldq: int,
                     num_pages: int, page_size: int, kcache, vcache, kscale, vscale, page_table, max_pages: int, lens,
                     O, ldo: int, lse=None, ws=None, ws_bytes: int | None = None, stream=None):
    """Attention of one token per sequence over the paged cache."""
    if ws_bytes is None:
        ws_bytes = _nbytes(ws)
    _check(_native.tern_attn_decode(x_type, kv_type, B, Hq, Hkv, D, scale, Q, ldq, num_pages, page_size, kcache,
                                    vcache, kscale, vscale, page_table, max_pages, lens, O, ldo,
                                    lse, ws, ws_bytes, _s(stream)), "tern_attn_decode")


def tern_rms_norm(x_type: int, in_type: int, T: int, H: int, K: int, X, ldx: int, res_type: int, R, ldr: int, S, lds: int,
                  W, w_add: float, eps: float, Y, ldy: int, stream=None):
    """Root-mean-square norm of T x H rows, with the residual's addition where R is given."""
    _check(_native.tern_rms_norm(x_type, in_type, T, H, K, X, ldx, res_type, R, ldr, S, lds, W, w_add, eps, Y, ldy,
                                 _s(stream)), "tern_rms_norm")


def tern_rms_norm_i8(x_type: int, in_type: int, M: int, K: int, X, ldx: int, res_type: int, R, ldr: int, S, lds: int, W,
                     w_add: float, eps: float, xq, a, stream=None):
    """The same with int8 codes and a factor per row, as tern_linear_i8 takes them."""
    _check(_native.tern_rms_norm_i8(x_type, in_type, M, K, X, ldx, res_type, R, ldr, S, lds, W, w_add, eps, xq, a,
                                    _s(stream)), "tern_rms_norm_i8")


def tern_attn_weights(x_type: int, kv_type: int, B: int, cu_q, Tq: int, Hq: int, Hkv: int, D: int, scale: float, Q, ldq: int,
                      lse, num_pages: int, page_size: int, kcache, kscale, page_table, max_pages: int, lens, known,
                      decay: float, weight, err=None, stream=None):
    """Add the attention weight that cached tokens receive from their sequences' newest rows."""
    _check(_native.tern_attn_weights(x_type, kv_type, B, cu_q, Tq, Hq, Hkv, D, scale, Q, ldq, lse, num_pages, page_size,
                                     kcache, kscale, page_table, max_pages, lens, known, decay, weight, err,
                                     _s(stream)), "tern_attn_weights")


def tern_kv_keep(B: int, Hkv: int, num_pages: int, page_size: int, weight, page_table, max_pages: int, lens, budget: int,
                 first: int, recent: int, keep, new_lens, stream=None):
    """Choose the tokens of each sequence and head that stay in the cache."""
    _check(_native.tern_kv_keep(B, Hkv, num_pages, page_size, weight, page_table, max_pages, lens, budget, first, recent,
                                keep, new_lens, _s(stream)), "tern_kv_keep")


def tern_kv_compact(kv_type: int, B: int, Hkv: int, D: int, num_pages: int, page_size: int, kcache, vcache, kscale, vscale,
                    weight, page_table, max_pages: int, keep, budget: int, to_table=None, to_pages: int = 0, err=None,
                    stream=None):
    """Move the kept tokens to the front of their sequence."""
    _check(_native.tern_kv_compact(kv_type, B, Hkv, D, num_pages, page_size, kcache, vcache, kscale, vscale, weight,
                                   page_table, max_pages, keep, budget, to_table, to_pages, err, _s(stream)),
           "tern_kv_compact")
