"""Python binding of the MI355X dense GEMM library (C ABI in include/dense_gemm_tile.h
and include/gemm_layer.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of libdense_gemm_tile_amd.so. Importing this package loads that
library and fails loudly if it has not been built (there is no CPU fallback). The
layer operators' calls convert their arguments in an extension module beside it
(csrc/binding.cpp), or in ctypes where that was not built for this interpreter.

Pointer arguments accept an int (a device address), None (NULL) or any object
with ``data_ptr()`` (a torch tensor). ``stream`` accepts an int (a hipStream_t
value), None (the default stream) or an object with a ``cuda_stream``
attribute (a torch stream).
"""
from __future__ import annotations

import ctypes
import os

# PyTorch brings a HIP runtime of its own, and of two runtimes in a process only
# the one that is loaded first finds the device: so PyTorch's comes first, in
# whichever order a program imports the two. Raw device addresses need no PyTorch,
# so one that is missing or does not load (whatever it raises) stops nothing here.
try:
    import torch as _torch  # noqa: F401
except Exception:
    pass

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libdense_gemm_tile_amd.so"
LIB_PATH = os.path.join(_PKG_DIR, LIB_NAME)

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_UNSUPPORTED = 2
GEMM_ERR_ALIAS = 3
GEMM_ERR_HIP = 4
GEMM_DTYPE_F16 = 0
GEMM_DTYPE_BF16 = 1
GEMM_DTYPE_F32_F16 = 2   # float32 A and B, rounded to f16 while staged
GEMM_DTYPE_F32_BF16 = 3  # float32 A and B, rounded to bf16 while staged
GEMM_DTYPE_F8_E4M3 = 4   # 8-bit float codes, OCP E4M3
GEMM_DTYPE_F8_E5M2 = 5   # 8-bit float codes, OCP E5M2
GEMM_DTYPE_F32 = 6       # float32 results and rows of the layer operators
GEMM_ACT_NONE, GEMM_ACT_RELU, GEMM_ACT_GELU, GEMM_ACT_GELU_ERF, GEMM_ACT_SILU = range(5)

# Every symbol the header declares, with its ctypes signature.
_i64, _int, _f32, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p
_SIGNATURES = {
    "gemm": (_int, [_i64, _i64, _i64, _int, _int, _int, _f32, _f32,
                    _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]),
    "gemm_validate": (_int, [_i64, _i64, _i64, _int, _int, _int, _f32, _f32,
                             _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64]),
    "gemm_i8": (_int, [_i64, _i64, _i64, _int, _int, ctypes.c_int32, ctypes.c_int32,
                       _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]),
    "gemm_i8_validate": (_int, [_i64, _i64, _i64, _int, _int, ctypes.c_int32, ctypes.c_int32,
                                _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64]),
    "gemm_last_error": (ctypes.c_char_p, []),
    "gemm_last_path": (ctypes.c_char_p, []),
    "gemm_tile_order": (_int, [_i64, _i64, _int, ctypes.POINTER(ctypes.c_int32),
                               ctypes.POINTER(ctypes.c_int32)]),
    # Layer operators.
    "gemm_linear": (_int, [_i64, _i64, _i64, _int, _int, _int, _vp, _i64, _vp, _i64, _vp, _int,
                           _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp]),
    "gemm_linear_validate": (_int, [_i64, _i64, _i64, _int, _int, _int, _vp, _i64, _vp, _i64, _vp,
                                    _int, _vp, _i64, _vp, _i64, _int, _vp, _i64]),
    "gemm_grouped": (_int, [_i64, _i64, _i64, _i64, _int, _int, _vp, _vp, _i64, _vp, _i64, _i64,
                            _vp, _int, _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp]),
    "gemm_grouped_validate": (_int, [_i64, _i64, _i64, _i64, _int, _int, _vp, _vp, _i64, _vp, _i64,
                                     _i64, _vp, _int, _vp, _i64, _vp, _i64, _int, _vp, _i64]),
    "gemm_grouped_grad_weight": (_int, [_i64, _i64, _i64, _i64, _int, _vp, _vp, _i64, _vp, _i64,
                                        _vp, _i64, _i64, _int, _int, _vp]),
    "gemm_grouped_grad_weight_validate": (_int, [_i64, _i64, _i64, _i64, _int, _vp, _vp, _i64, _vp,
                                                 _i64, _vp, _i64, _i64, _int, _int]),
    "gemm_act_grad": (_int, [_i64, _i64, _i64, _int, _int, _vp, _vp, _i64, _vp, _i64, _vp, _i64,
                             _vp, _vp, _i64, _vp]),
    "gemm_act_grad_workspace": (_i64, [_i64, _i64, _i64]),
    "gemm_route": (_int, [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp]),
    "gemm_route_workspace": (_i64, [_i64, _i64, _i64]),
    "gemm_dispatch": (_int, [_i64, _i64, _i64, _int, _vp, _i64, _vp, _vp, _i64, _vp]),
    "gemm_combine": (_int, [_i64, _i64, _i64, _int, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64,
                            _vp]),
    "gemm_combine_grad": (_int, [_i64, _i64, _i64, _int, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64,
                                 _vp, _vp]),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built. Build it with `python dense_gemm_tile_amd/build.py` "
            "(hipcc, gfx950); this package has no CPU fallback.")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


class GemmError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"gemm failed with status {code}: {message}")
        self.code = code


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


_DTYPE_CODES = {"f16": GEMM_DTYPE_F16, "bf16": GEMM_DTYPE_BF16, "f32_f16": GEMM_DTYPE_F32_F16,
                "f32_bf16": GEMM_DTYPE_F32_BF16, "f8e4m3": GEMM_DTYPE_F8_E4M3,
                "f8e5m2": GEMM_DTYPE_F8_E5M2, "f32": GEMM_DTYPE_F32}
_ACT_CODES = {"none": GEMM_ACT_NONE, "relu": GEMM_ACT_RELU, "gelu": GEMM_ACT_GELU,
              "gelu_erf": GEMM_ACT_GELU_ERF, "silu": GEMM_ACT_SILU}


def _dtype(d):
    if isinstance(d, str):
        return _DTYPE_CODES[d]
    return int(d)


def _act(a):
    if isinstance(a, str):
        return _ACT_CODES[a]
    return int(a)


class _CtypesCalls:
    """The calls of the extension module (_binding) through ctypes: the same arguments and status
    codes, at about 3 us of host time a call instead of 0.8."""

    # Positions of dtypes, and of the activation, among an entry point's arguments.
    _DTYPES = {"gemm_linear": (3, 16), "gemm_grouped": (4, 18), "gemm_grouped_grad_weight": (4, 13),
               "gemm_act_grad": (3,), "gemm_dispatch": (3,), "gemm_combine": (3,), "gemm_combine_grad": (3,)}
    _ACT = {"gemm_linear": 11, "gemm_grouped": 13, "gemm_act_grad": 4}

    def __getattr__(self, name):  # once a name
        fn, types = getattr(_lib, name), _SIGNATURES[name][1]
        convert = [_ptr if t is _vp else (lambda v: v) for t in types]
        if types[-1] is _vp:
            convert[-1] = _stream
        for i in self._DTYPES.get(name, ()):
            convert[i] = _dtype
        if name in self._ACT:
            convert[self._ACT[name]] = _act
        call = lambda *args: fn(*[c(a) for c, a in zip(convert, args, strict=True)])  # noqa: E731
        setattr(self, name, call)
        return call


# Calls of the layer operators that enqueue work: through the extension module, or
# through ctypes where it was not built for this interpreter.
try:
    from . import _binding as _fast
except ImportError:
    _fast = _CtypesCalls()


def _check(st: int) -> None:
    if st != GEMM_OK:
        raise GemmError(st, gemm_last_error())


def gemm(M, N, K, dtype, transA, transB, alpha, beta, A, lda, B, ldb, C, ldc, D, ldd,
         stream=None):
    """Enqueue D = alpha*op(A)@op(B) + beta*C; raises GemmError on a non-zero status."""
    st = _lib.gemm(M, N, K, _dtype(dtype), int(transA), int(transB), alpha, beta,
                   _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, _ptr(D), ldd, _stream(stream))
    if st != GEMM_OK:
        raise GemmError(st, gemm_last_error())


def gemm_status(M, N, K, dtype, transA, transB, alpha, beta, A, lda, B, ldb, C, ldc, D, ldd,
                stream=None) -> int:
    """Same as gemm() but returns the status code instead of raising."""
    return _lib.gemm(M, N, K, _dtype(dtype), int(transA), int(transB), alpha, beta,
                     _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, _ptr(D), ldd, _stream(stream))


def gemm_validate(M, N, K, dtype, transA, transB, alpha, beta, A, lda, B, ldb, C, ldc, D,
                  ldd) -> int:
    """Host-only checks and path selection; returns the status code."""
    return _lib.gemm_validate(M, N, K, _dtype(dtype), int(transA), int(transB), alpha, beta,
                              _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, _ptr(D), ldd)


def gemm_i8(M, N, K, transA, transB, alpha, beta, A, lda, B, ldb, C, ldc, D, ldd, stream=None):
    """Enqueue the int8 form D = alpha*op(A)@op(B) + beta*C (int32 C/D, integer
    alpha/beta, int32 wraparound); raises GemmError on a non-zero status."""
    st = _lib.gemm_i8(M, N, K, int(transA), int(transB), int(alpha), int(beta), _ptr(A), lda,
                      _ptr(B), ldb, _ptr(C), ldc, _ptr(D), ldd, _stream(stream))
    if st != GEMM_OK:
        raise GemmError(st, gemm_last_error())


def gemm_i8_validate(M, N, K, transA, transB, alpha, beta, A, lda, B, ldb, C, ldc, D,
                     ldd) -> int:
    """Host-only checks of the int8 form; returns the status code."""
    return _lib.gemm_i8_validate(M, N, K, int(transA), int(transB), int(alpha), int(beta),
                                 _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, _ptr(D), ldd)


def gemm_linear(M, N, K, dtype, transA, transB, A, lda, B, ldb, bias, act, R, ldr, Y, ldy,
                out_dtype, Z=None, ldz=0, stream=None):
    """Enqueue Z = op(A)@op(B) + bias, Y = act(Z) + R (bias, R and Z may be None); act is one of
    "none", "relu", "gelu", "gelu_erf", "silu"; raises GemmError on a non-zero status."""
    _check(_fast.gemm_linear(M, N, K, dtype, transA, transB, A, lda, B, ldb, bias, act, R, ldr, Y,
                             ldy, out_dtype, Z, ldz, stream))


def gemm_linear_validate(M, N, K, dtype, transA, transB, A, lda, B, ldb, bias, act, R, ldr, Y, ldy,
                         out_dtype, Z=None, ldz=0) -> int:
    """Host-only checks and kernel choice of gemm_linear(); returns the status code."""
    return _lib.gemm_linear_validate(M, N, K, _dtype(dtype), int(transA), int(transB), _ptr(A),
                                     lda, _ptr(B), ldb, _ptr(bias), _act(act), _ptr(R), ldr,
                                     _ptr(Y), ldy, _dtype(out_dtype), _ptr(Z), ldz)


def gemm_grouped(G, M, N, K, dtype, transB, offsets, A, lda, B, ldb, stride_b, bias, act, R, ldr,
                 Y, ldy, out_dtype, Z=None, ldz=0, stream=None):
    """Enqueue gemm_linear() with one B and bias per group of rows offsets[g] .. offsets[g+1]-1."""
    _check(_fast.gemm_grouped(G, M, N, K, dtype, transB, offsets, A, lda, B, ldb, stride_b, bias,
                              act, R, ldr, Y, ldy, out_dtype, Z, ldz, stream))


def gemm_grouped_validate(G, M, N, K, dtype, transB, offsets, A, lda, B, ldb, stride_b, bias, act,
                          R, ldr, Y, ldy, out_dtype, Z=None, ldz=0) -> int:
    """Host-only checks and kernel choice of gemm_grouped(); returns the status code."""
    return _lib.gemm_grouped_validate(G, M, N, K, _dtype(dtype), int(transB), _ptr(offsets),
                                      _ptr(A), lda, _ptr(B), ldb, stride_b, _ptr(bias), _act(act),
                                      _ptr(R), ldr, _ptr(Y), ldy, _dtype(out_dtype), _ptr(Z), ldz)


def gemm_grouped_grad_weight(G, M, N, K, dtype, offsets, A, lda, B, ldb, D, ldd, stride_d,
                             out_dtype, accumulate=False, stream=None):
    """Enqueue D_g = A_g^T @ B_g (+ D_g when accumulate) over the rows of each group."""
    _check(_fast.gemm_grouped_grad_weight(G, M, N, K, dtype, offsets, A, lda, B, ldb, D, ldd,
                                          stride_d, out_dtype, accumulate, stream))


def gemm_grouped_grad_weight_validate(G, M, N, K, dtype, offsets, A, lda, B, ldb, D, ldd, stride_d,
                                      out_dtype, accumulate=False) -> int:
    """Host-only checks of gemm_grouped_grad_weight(); returns the status code."""
    return _lib.gemm_grouped_grad_weight_validate(G, M, N, K, _dtype(dtype), _ptr(offsets),
                                                  _ptr(A), lda, _ptr(B), ldb, _ptr(D), ldd,
                                                  stride_d, _dtype(out_dtype), int(accumulate))


def gemm_act_grad(G, M, N, dtype, act, offsets, dY, lddy, Z, ldz, dZ, lddz, db, workspace,
                  workspace_bytes, stream=None):
    """Enqueue dZ = dY * act'(Z) and db[g] = the sum of dZ over each group's rows (float32).
    offsets None: one group. workspace: gemm_act_grad_workspace(G, M, N) bytes on the device."""
    _check(_fast.gemm_act_grad(G, M, N, dtype, act, offsets, dY, lddy, Z, ldz, dZ, lddz, db,
                               workspace, workspace_bytes, stream))


def gemm_act_grad_workspace(G, M, N) -> int:
    """Bytes of workspace that gemm_act_grad() needs."""
    return _fast.gemm_act_grad_workspace(G, M, N)


def gemm_route(T, top, E, ids, offsets, order, slot, workspace, workspace_bytes, stream=None):
    """Enqueue the stable sort of T x top int32 expert ids: offsets[E + 1], order[T * top] and
    slot[T * top] (int32). workspace: gemm_route_workspace(T, top, E) bytes on the device."""
    _check(_fast.gemm_route(T, top, E, ids, offsets, order, slot, workspace, workspace_bytes,
                            stream))


def gemm_route_workspace(T, top, E) -> int:
    """Bytes of workspace that gemm_route() needs."""
    return _fast.gemm_route_workspace(T, top, E)


def gemm_dispatch(T, top, H, dtype, X, ldx, slot, Xs, ldxs, stream=None):
    """Enqueue Xs[slot[t][j]] = X[t] ("f16", "bf16" or "f32" rows of H values)."""
    _check(_fast.gemm_dispatch(T, top, H, dtype, X, ldx, slot, Xs, ldxs, stream))


def gemm_combine(T, top, H, dtype, Ys, ldys, slot, weights, R, ldr, Y, ldy, stream=None):
    """Enqueue Y[t] = sum_j weights[t][j] * Ys[slot[t][j]] + R[t] (weights float32 or None for
    ones, R may be None)."""
    _check(_fast.gemm_combine(T, top, H, dtype, Ys, ldys, slot, weights, R, ldr, Y, ldy, stream))


def gemm_combine_grad(T, top, H, dtype, dY, lddy, Ys, ldys, slot, weights, dYs, lddys, dweights,
                      stream=None):
    """Enqueue dYs[slot[t][j]] = weights[t][j] * dY[t] and dweights[t][j] = <dY[t], Ys[slot]>."""
    _check(_fast.gemm_combine_grad(T, top, H, dtype, dY, lddy, Ys, ldys, slot, weights, dYs, lddys,
                                   dweights, stream))


def gemm_last_error() -> str:
    return _lib.gemm_last_error().decode()


def gemm_last_path() -> str:
    return _lib.gemm_last_path().decode()


def gemm_tile_order(tiles_m: int, tiles_n: int, group_m: int):
    """The scheduler's workgroup -> (tile row, tile column) map, as two lists."""
    n = tiles_m * tiles_n
    tm = (ctypes.c_int32 * max(n, 1))()
    tn = (ctypes.c_int32 * max(n, 1))()
    st = _lib.gemm_tile_order(tiles_m, tiles_n, group_m, tm, tn)
    if st != GEMM_OK:
        raise GemmError(st, gemm_last_error())
    return list(tm[:n]), list(tn[:n])


__all__ = ["gemm_i8", "gemm_i8_validate", "gemm", "gemm_status", "gemm_validate", "gemm_last_error", "gemm_last_path",
           "gemm_tile_order", "GemmError", "GEMM_OK", "GEMM_ERR_INVALID_ARG",
           "GEMM_ERR_UNSUPPORTED", "GEMM_ERR_ALIAS", "GEMM_ERR_HIP", "GEMM_DTYPE_F16",
           "GEMM_DTYPE_BF16", "GEMM_DTYPE_F32_F16", "GEMM_DTYPE_F32_BF16", "GEMM_DTYPE_F8_E4M3",
           "GEMM_DTYPE_F8_E5M2", "LIB_PATH",
           "gemm_linear", "gemm_linear_validate", "gemm_grouped", "gemm_grouped_validate",
           "gemm_grouped_grad_weight", "gemm_grouped_grad_weight_validate", "gemm_act_grad",
           "gemm_act_grad_workspace", "gemm_route", "gemm_route_workspace", "gemm_dispatch",
           "gemm_combine", "gemm_combine_grad", "GEMM_DTYPE_F32", "GEMM_ACT_NONE",
           "GEMM_ACT_RELU", "GEMM_ACT_GELU", "GEMM_ACT_GELU_ERF", "GEMM_ACT_SILU"]
