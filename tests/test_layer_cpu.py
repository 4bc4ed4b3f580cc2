"""Host-side tests of the layer operators: refusals, aliasing rules, empty calls, workspace sizes
and kernel choice. Nothing here launches a kernel; pointers are fake addresses that the library only
compares."""
import ctypes
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A0, B0, Y0, R0, Z0, P0 = (0x10000000 * i for i in range(1, 7))
W0 = 0x70000000


@pytest.fixture(scope="module")
def lib():
    so = os.path.join(ROOT, "dense_gemm_tile_amd", "libdense_gemm_tile_amd.so")
    if not os.path.exists(so):
        subprocess.run([sys.executable, os.path.join(ROOT, "dense_gemm_tile_amd", "build.py")], check=True)
    import dense_gemm_tile_amd as dgt
    return dgt


def linear(lib, M=64, N=64, K=64, dtype=1, tA=0, tB=1, A=A0, lda=None, B=B0, ldb=None, bias=None, act=0, R=None,
           ldr=None, Y=Y0, ldy=None, out=None, Z=None, ldz=None):
    return lib.gemm_linear_validate(M, N, K, dtype, tA, tB, A, (M if tA else K) if lda is None else lda, B,
                                    (K if tB else N) if ldb is None else ldb, bias, act, R, N if ldr is None else ldr,
                                    Y, N if ldy is None else ldy, dtype if out is None else out, Z,
                                    N if ldz is None else ldz)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(M=1 << 31), 2), (dict(dtype=2), 2), (dict(dtype=6), 2),
    (dict(dtype=-1), 2), (dict(out=0), 2), (dict(out=5), 2), (dict(act=5), 1), (dict(act=-1), 1), (dict(lda=63), 1),
    (dict(tA=1, lda=63), 1), (dict(ldb=63), 1), (dict(tB=0, ldb=63), 1), (dict(ldy=63), 1),
    (dict(R=R0, ldr=63), 1), (dict(Z=Z0, ldz=63), 1), (dict(A=None), 1), (dict(B=None), 1), (dict(Y=None), 1),
    (dict(A=A0 + 1), 1), (dict(Y=Y0 + 1), 1), (dict(out=6, Y=Y0 + 2), 1), (dict(bias=P0 + 1), 1), (dict(R=R0 + 1), 1),
    (dict(Z=Z0 + 1), 1), (dict(Y=A0), 3), (dict(Y=B0 + 2), 3), (dict(Z=A0), 3), (dict(Z=Y0), 3), (dict(bias=Y0 + 8), 3),
    (dict(R=Y0 + 4), 3), (dict(R=Y0, ldr=65), 3), (dict(R=R0, Z=R0), 3),
])
def test_linear_refusals(lib, kw, code):
    assert linear(lib, **kw) == code
    assert lib.gemm_last_error()


@pytest.mark.parametrize("kw", [
    dict(), dict(R=Y0), dict(R=R0, bias=P0, Z=Z0, act=4), dict(out=6), dict(K=0, A=None, B=None, lda=1, ldb=1), dict(M=0, Y=None),
    dict(N=0, Y=None, A=None, ldy=1), dict(M=1, N=1, K=1), dict(tA=1, tB=0), dict(A=A0 + 2), dict(lda=65),
])
def test_linear_accepts(lib, kw):
    assert linear(lib, **kw) == 0, lib.gemm_last_error()
    assert lib.gemm_last_error() == ""
    path = lib.gemm_last_path()
    assert path.startswith("linear mfma" if kw.get("M", 1) and kw.get("N", 1) else "noop")


def test_linear_path_names_the_epilogue(lib):
    assert linear(lib, R=R0, bias=P0, Z=Z0, act=2, out=6) == 0
    for word in ("linear", "NT", "act=gelu", "bias", "residual", " z", "f32-out"):
        assert word in lib.gemm_last_path()


def grouped(lib, G=4, M=64, N=64, K=64, dtype=1, tB=1, off=P0, A=A0, lda=None, B=B0, ldb=None, stride=None, bias=None,
            act=0, R=None, ldr=None, Y=Y0, ldy=None, out=None, Z=None):
    return lib.gemm_grouped_validate(G, M, N, K, dtype, tB, off, A, K if lda is None else lda, B,
                                     (K if tB else N) if ldb is None else ldb, N * K if stride is None else stride,
                                     bias, act, R, N if ldr is None else ldr, Y, N if ldy is None else ldy,
                                     dtype if out is None else out, Z, N)


@pytest.mark.parametrize("kw,code", [
    (dict(G=-1), 1), (dict(G=65536), 2), (dict(M=-1), 1), (dict(off=None), 1), (dict(off=P0 + 2), 1), (dict(off=Y0), 3),
    (dict(stride=-1), 1), (dict(lda=63), 1), (dict(ldb=63), 1), (dict(A=None), 1), (dict(B=None), 1), (dict(act=9), 1),
    (dict(dtype=4), 2), (dict(Y=B0 + 3 * 64 * 64 * 2), 3), (dict(bias=Y0), 3), (dict(Z=P0), 3),
])
def test_grouped_refusals(lib, kw, code):
    assert grouped(lib, **kw) == code
    assert lib.gemm_last_error()


@pytest.mark.parametrize("kw", [dict(), dict(G=0), dict(M=0, A=None, Y=None), dict(stride=0), dict(K=0, A=None, B=None, lda=1, ldb=1),
                                dict(G=1, stride=-5), dict(bias=W0, R=Y0, act=4)])
def test_grouped_accepts(lib, kw):
    assert grouped(lib, **kw) == 0, lib.gemm_last_error()


def grad_weight(lib, G=4, M=64, N=64, K=64, dtype=1, off=P0, A=A0, lda=64, B=B0, ldb=64, D=Y0, ldd=64, stride=64 * 64,
                out=None, acc=0):
    return lib.gemm_grouped_grad_weight_validate(G, M, N, K, dtype, off, A, lda, B, ldb, D, ldd, stride,
                                                 dtype if out is None else out, acc)


@pytest.mark.parametrize("kw,code", [
    (dict(G=-1), 1), (dict(G=1 << 20), 2), (dict(N=-2), 1), (dict(stride=64 * 64 - 1), 1), (dict(ldd=63), 1),
    (dict(lda=63), 1), (dict(ldb=63), 1), (dict(D=None), 1), (dict(off=None), 1), (dict(D=A0 + 2), 3), (dict(D=P0), 3),
    (dict(out=3), 2), (dict(dtype=3), 2),
])
def test_grad_weight_refusals(lib, kw, code):
    assert grad_weight(lib, **kw) == code


@pytest.mark.parametrize("kw", [dict(), dict(M=0, A=None, B=None), dict(G=0, stride=0), dict(N=0), dict(out=6, acc=1),
                                dict(G=1, stride=0)])
def test_grad_weight_accepts(lib, kw):
    assert grad_weight(lib, **kw) == 0, lib.gemm_last_error()


def call(lib, name, *args):
    """The status of an entry point that would launch if it accepted its arguments: only refused
    and empty calls are made here."""
    return getattr(lib._lib, name)(*args)


def act_grad(lib, G=1, M=64, N=64, dtype=1, act=2, off=None, dY=A0, lddy=64, Z=Z0, ldz=64, dZ=Y0, lddz=64, db=R0,
             ws=W0, size=None):
    need = lib.gemm_act_grad_workspace(G, M, N)
    return call(lib, "gemm_act_grad", G, M, N, dtype, act, off, dY, lddy, Z, ldz, dZ, lddz, db, ws,
                need if size is None else size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(G=-1), 1), (dict(G=2), 1), (dict(G=70000, off=P0), 2), (dict(M=-1), 1), (dict(dtype=6), 2), (dict(act=7), 1),
    (dict(lddy=63), 1), (dict(ldz=63), 1), (dict(lddz=63), 1), (dict(dY=None), 1), (dict(Z=None), 1), (dict(size=0), 1),
    (dict(ws=None), 1), (dict(ws=W0 + 8), 1), (dict(db=R0 + 2), 1), (dict(dZ=A0 + 2), 3), (dict(dZ=A0, lddz=72), 3),
    (dict(db=A0), 3), (dict(db=Y0), 3), (dict(ws=A0), 3), (dict(ws=Y0), 3), (dict(ws=R0), 3), (dict(off=Y0), 3),
    (dict(off=P0 + 1), 1),
])
def test_act_grad_refusals(lib, kw, code):
    assert act_grad(lib, **kw) == code
    assert lib.gemm_last_error()


@pytest.mark.parametrize("kw", [dict(N=0), dict(G=0, off=P0), dict(M=0, db=None), dict(dZ=None, db=None)])
def test_act_grad_empty(lib, kw):
    assert act_grad(lib, **kw) == 0, lib.gemm_last_error()
    assert lib.gemm_last_path().startswith("noop")


def route(lib, T=8, top=2, E=4, ids=A0, off=B0, order=Y0, slot=R0, ws=W0, size=1 << 30):
    return call(lib, "gemm_route", T, top, E, ids, off, order, slot, ws, size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(top=-1), 1), (dict(E=-1), 1), (dict(E=1025), 2), (dict(T=1 << 30, top=4), 2),
    (dict(ids=None), 1), (dict(off=None), 1), (dict(order=None), 1), (dict(slot=None), 1), (dict(ids=A0 + 1), 1),
    (dict(off=A0), 3), (dict(order=A0 + 4), 3), (dict(slot=Y0), 3), (dict(T=100000, size=4), 1),
    (dict(T=100000, ws=None), 1), (dict(T=100000, ws=A0), 3),
])
def test_route_refusals(lib, kw, code):
    assert route(lib, **kw) == code
    assert lib.gemm_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(H=-1), 1), (dict(dtype=2), 2), (dict(ldx=63), 1), (dict(ldxs=63), 1), (dict(X=None), 1),
    (dict(slot=None), 1), (dict(Xs=None), 1), (dict(X=A0 + 1), 1), (dict(Xs=A0 + 64), 3), (dict(Xs=R0), 3),
])
def test_dispatch_refusals(lib, kw, code):
    d = dict(T=8, top=2, H=64, dtype=1, X=A0, ldx=64, slot=R0, Xs=Y0, ldxs=64) | kw
    assert call(lib, "gemm_dispatch", *d.values(), None) == code
    assert lib.gemm_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(top=-1), 1), (dict(dtype=3), 2), (dict(ldys=63), 1), (dict(ldr=63), 1), (dict(ldy=63), 1), (dict(Ys=None), 1),
    (dict(slot=None), 1), (dict(Y=None), 1), (dict(w=P0 + 2), 1), (dict(Y=A0), 3), (dict(Y=R0), 3), (dict(Y=P0), 3),
    (dict(R=Y0 + 2), 3), (dict(R=Y0, ldr=72), 3),
])
def test_combine_refusals(lib, kw, code):
    d = dict(T=8, top=2, H=64, dtype=1, Ys=A0, ldys=64, slot=R0, w=P0, R=Z0, ldr=64, Y=Y0, ldy=64) | kw
    assert call(lib, "gemm_combine", *d.values(), None) == code
    assert lib.gemm_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(H=-1), 1), (dict(dtype=5), 2), (dict(lddy=63), 1), (dict(ldys=63), 1), (dict(lddys=63), 1),
    (dict(dY=None), 1), (dict(Ys=None), 1), (dict(slot=None), 1), (dict(dYs=B0 + 2), 3), (dict(dYs=A0), 3),
    (dict(dw=B0), 3), (dict(dw=P0), 3), (dict(dw=Y0), 3), (dict(dYs=B0, lddys=72), 3),
])
def test_combine_grad_refusals(lib, kw, code):
    d = dict(T=8, top=2, H=64, dtype=1, dY=A0, lddy=64, Ys=B0, ldys=64, slot=R0, w=P0, dYs=Y0, lddys=64, dw=Z0) | kw
    assert call(lib, "gemm_combine_grad", *d.values(), None) == code
    assert lib.gemm_last_error()


def test_empty_row_calls(lib):
    for T, H in ((0, 64), (8, 0)):
        assert call(lib, "gemm_dispatch", T, 2, H, 1, A0, 64, R0, Y0, 64, None) == 0
        assert call(lib, "gemm_combine", T, 2, H, 1, A0, 64, R0, None, None, 0, Y0, 64, None) == 0
    assert call(lib, "gemm_combine_grad", 0, 2, 64, 1, A0, 64, B0, 64, R0, None, Y0, 64, Z0, None) == 0
    assert call(lib, "gemm_combine_grad", 8, 2, 64, 1, A0, 64, B0, 64, R0, None, None, 0, None, None) == 0


def test_workspace_sizes(lib):
    assert lib.gemm_route_workspace(0, 4, 8) == 0
    assert lib.gemm_route_workspace(32, 4, 64) == 0
    assert lib.gemm_route_workspace(1 << 20, 8, 64) >= 65 * 4
    assert lib.gemm_route_workspace(-1, 4, 8) == 0 and lib.gemm_route_workspace(8, 4, 5000) == 0
    assert lib.gemm_act_grad_workspace(3, 100, 64) >= 4 * 64 * 4
    assert lib.gemm_act_grad_workspace(1, -1, 64) == 0
    # far past 64 bits of bytes, or refused: no size that is too small
    big = lib.gemm_act_grad_workspace(65535, 2 ** 31 - 1024, 2 ** 31 - 1024)
    assert big == 0 or big > 2 ** 50


def test_unknown_names_raise(lib):
    with pytest.raises(KeyError):
        lib.gemm_linear(1, 1, 1, "bf16", 0, 1, A0, 1, B0, 1, None, "swish", None, 0, Y0, 1, "bf16")
    with pytest.raises(KeyError):
        lib.gemm_linear(1, 1, 1, "int3", 0, 1, A0, 1, B0, 1, None, "none", None, 0, Y0, 1, "bf16")
    with pytest.raises(lib.GemmError):
        lib.gemm_linear(1, 1, 1, "bf16", 0, 1, A0, 1, B0, 1, None, "none", None, 0, A0, 1, "bf16")


def test_forced_tile_must_exist(lib, monkeypatch):
    env = ctypes.CDLL(None)
    env.setenv(b"GEMM_LAYER_TILE", b"t1x1", 1)
    try:
        assert linear(lib) == 1
    finally:
        env.unsetenv(b"GEMM_LAYER_TILE")
    assert linear(lib) == 0
