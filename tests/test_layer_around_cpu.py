"""Refusals of the operators around a layer: norms, the gate, products with 4-bit weights, the loss.
Nothing here launches a kernel: every call is refused or does nothing, and pointers are fake addresses
that the library only compares. Through the extension module and through ctypes."""
import math

import pytest

import dense_gemm_tile_amd as dgt

P = [0x100000000 * (i + 1) for i in range(12)]
CALLS = [dgt._binding if hasattr(dgt, "_binding") else dgt._fast, dgt._CtypesCalls()]


def status(name, args):
    found = {c.__class__.__name__: getattr(c, name)(*args) for c in CALLS}
    assert len(set(found.values())) == 1, found
    return next(iter(found.values()))


def norm(M=4, N=64, dtype="bf16", X=P[0], ldx=64, gamma=P[1], beta=P[2], eps=1e-5, Y=P[3], ldy=64, mean=P[4], rstd=P[5]):
    return status("gemm_norm", (M, N, dtype, X, ldx, gamma, beta, eps, Y, ldy, mean, rstd, None))


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(N=0), 1), (dict(M=1 << 31), 2), (dict(N=1 << 31, ldx=1 << 31, ldy=1 << 31), 2),
    (dict(dtype=2), 2), (dict(dtype=7), 2), (dict(ldx=63), 1), (dict(ldy=63), 1), (dict(eps=-1e-9), 1), (dict(eps=math.nan), 1),
    (dict(eps=math.inf), 1), (dict(X=None), 1), (dict(Y=None), 1), (dict(X=P[0] + 1), 1), (dict(dtype="f32", Y=P[3] + 2), 1),
    (dict(gamma=P[1] + 1), 1), (dict(beta=P[2] + 1), 1), (dict(mean=P[4] + 2), 1), (dict(rstd=P[5] + 1), 1),
    (dict(Y=P[0] + 64), 3), (dict(Y=P[0], ldy=65), 3), (dict(Y=P[1] - 64), 3), (dict(Y=P[2] + 8), 3), (dict(mean=P[0]), 3),
    (dict(rstd=P[3] + 64), 3), (dict(rstd=P[4] + 12), 3), (dict(mean=P[1]), 3), (dict(M=0), 0), (dict(M=0, X=None, Y=None), 0)])
def test_norm(kw, code):
    assert norm(**kw) == code, dgt.gemm_last_error()


def norm_grad(M=4, N=64, dtype="bf16", dY=P[0], lddy=64, X=P[1], ldx=64, gamma=P[2], mean=P[3], rstd=P[4], R=P[5], ldr=64,
              dX=P[6], lddx=64, dgamma=P[7], dbeta=P[8], ws=P[9], size=None):
    need = dgt.gemm_norm_grad_workspace(M, N)
    return status("gemm_norm_grad", (M, N, dtype, dY, lddy, X, ldx, gamma, mean, rstd, R, ldr, dX, lddx, dgamma, dbeta, ws,
                                     need if size is None else size, None))


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(N=0), 1), (dict(M=1 << 31), 2), (dict(dtype=4), 2), (dict(lddy=63), 1), (dict(ldx=63), 1),
    (dict(ldr=63), 1), (dict(lddx=63), 1), (dict(dY=None), 1), (dict(X=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1),
    (dict(dY=P[0] + 1), 1), (dict(dgamma=P[7] + 2), 1), (dict(ws=None), 1), (dict(ws=P[9] + 8), 1), (dict(size=10), 1),
    (dict(dX=P[0] + 2), 3), (dict(dX=P[0], lddx=65), 3), (dict(dX=P[2]), 3), (dict(dX=P[3]), 3), (dict(dgamma=P[0]), 3),
    (dict(dgamma=P[8] + 4), 3), (dict(dbeta=P[6]), 3), (dict(ws=P[1]), 3), (dict(ws=P[6] + 16), 3), (dict(ws=P[7]), 3),
    (dict(dX=None, dgamma=None, dbeta=None), 0), (dict(M=0, dgamma=None, dbeta=None, ws=None), 0)])
def test_norm_grad(kw, code):
    assert norm_grad(**kw) == code, dgt.gemm_last_error()


def gate(T=4, E=64, top=4, dtype="f32", L=P[0], ldl=64, score="softmax", bias=P[1], groups=1, top_groups=1, group_top=1,
         renorm=1, scale=1.0, ids=P[2], weights=P[3]):
    return status("gemm_gate", (T, E, top, dtype, L, ldl, score, bias, groups, top_groups, group_top, renorm, scale, ids,
                                weights, None))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(E=-1), 1), (dict(top=-1), 1), (dict(T=1 << 31), 2), (dict(T=1 << 30, top=4), 2),
    (dict(E=1025, ldl=1025), 2), (dict(E=128, ldl=128, top=65), 2), (dict(E=3, ldl=3), 1), (dict(dtype=3), 2), (dict(ldl=63), 1),
    (dict(score=2), 1), (dict(score=-1), 1), (dict(groups=0), 1), (dict(groups=5), 1), (dict(groups=-8), 1),
    (dict(groups=8, top_groups=0), 1), (dict(groups=8, top_groups=9), 1), (dict(groups=8, top_groups=4, group_top=3), 1),
    (dict(groups=8, top_groups=4, group_top=0), 1), (dict(group_top=3), 1), (dict(groups=64, top_groups=8, group_top=2), 1),
    (dict(groups=32, top_groups=1, top=3), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(L=None), 1),
    (dict(L=P[0] + 2), 1), (dict(bias=P[1] + 2), 1), (dict(ids=None), 1), (dict(weights=None), 1), (dict(ids=P[2] + 2), 1),
    (dict(ids=P[0]), 3), (dict(weights=P[0] + 1020), 3), (dict(weights=P[1]), 3), (dict(weights=P[2] + 60), 3),
    (dict(T=0), 0), (dict(top=0), 0), (dict(T=0, L=None, ids=None, weights=None), 0), (dict(E=0, top=0, ldl=1), 0)])
def test_gate(kw, code):
    assert gate(**kw) == code, dgt.gemm_last_error()


def gate_grad(T=4, E=64, top=4, dtype="f32", L=P[0], ldl=64, score="sigmoid", renorm=1, scale=1.0, ids=P[1], dw=P[2], dL=P[3],
              lddl=64):
    return status("gemm_gate_grad", (T, E, top, dtype, L, ldl, score, renorm, scale, ids, dw, dL, lddl, None))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(E=1025, ldl=1025, lddl=1025), 2), (dict(top=65), 2), (dict(dtype=5), 2), (dict(ldl=63), 1),
    (dict(lddl=63), 1), (dict(score=7), 1), (dict(scale=-math.inf), 1), (dict(L=None), 1), (dict(dL=None), 1),
    (dict(ids=None), 1), (dict(dw=None), 1), (dict(dL=P[3] + 1), 1), (dict(dL=P[0] + 4), 3), (dict(dL=P[0], lddl=65), 3),
    (dict(dL=P[1]), 3), (dict(dL=P[2] + 4), 3), (dict(T=0), 0), (dict(E=0, ldl=1, lddl=1), 0)])
def test_gate_grad(kw, code):
    assert gate_grad(**kw) == code, dgt.gemm_last_error()


def linear_w4(M=4, N=64, K=128, dtype="bf16", A=P[0], lda=128, B=P[1], ldb=128, scales=P[2], zeros=P[3], lds=4, group=32,
              bias=P[4], act="silu", R=P[5], ldr=64, Y=P[6], ldy=64, out="bf16"):
    return status("gemm_linear_w4", (M, N, K, dtype, A, lda, B, ldb, scales, zeros, lds, group, bias, act, R, ldr, Y, ldy, out,
                                     None))


BAD_W4 = [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(M=1 << 31), 2), (dict(dtype="f32"), 2), (dict(dtype=4), 2),
    (dict(out="f16"), 2), (dict(act=5), 1), (dict(group=0), 1), (dict(group=16), 1), (dict(group=33), 1), (dict(group=-32), 1),
    (dict(lda=127), 1), (dict(ldb=126), 1), (dict(ldb=129), 1), (dict(lds=3), 1), (dict(ldr=63), 1), (dict(ldy=63), 1),
    (dict(A=None), 1), (dict(B=None), 1), (dict(scales=None), 1), (dict(Y=None), 1), (dict(A=P[0] + 1), 1),
    (dict(scales=P[2] + 1), 1), (dict(zeros=P[3] + 1), 1), (dict(bias=P[4] + 1), 1), (dict(R=P[5] + 1), 1),
    (dict(out="f32", Y=P[6] + 2), 1), (dict(Y=P[0]), 3), (dict(Y=P[1] + 64), 3), (dict(Y=P[2]), 3), (dict(Y=P[3] + 2), 3),
    (dict(Y=P[4]), 3), (dict(Y=P[5] + 2), 3), (dict(Y=P[5], ldy=65), 3), (dict(M=0), 0), (dict(N=0), 0)]


@pytest.mark.parametrize("kw,code", BAD_W4 + [(dict(M=2 ** 31 - 2048, N=2 ** 31 - 2048, ldr=2 ** 31, ldy=2 ** 31, R=None,
                                                    bias=None, A=0x10, K=1, lda=1, Y=1 << 62, zeros=None, B=1 << 40,
                                                    scales=1 << 50), 2)])
def test_linear_w4(kw, code):
    assert linear_w4(**kw) == code, dgt.gemm_last_error()


def grouped_w4(G=3, M=4, N=64, K=128, dtype="bf16", offsets=P[7], A=P[0], lda=128, B=P[1], ldb=128, stride_b=128 * 64,
               scales=P[2], zeros=P[3], lds=4, stride_s=256, group=32, bias=P[4], act="silu", R=P[5], ldr=64, Y=P[6], ldy=64,
               out="bf16"):
    return status("gemm_grouped_w4", (G, M, N, K, dtype, offsets, A, lda, B, ldb, stride_b, scales, zeros, lds, stride_s, group,
                                      bias, act, R, ldr, Y, ldy, out, None))


@pytest.mark.parametrize("kw,code", BAD_W4 + [
    (dict(G=-1), 1), (dict(G=65536), 2), (dict(stride_b=-2), 1), (dict(stride_b=8191), 1), (dict(stride_s=-1), 1),
    (dict(offsets=None), 1), (dict(offsets=P[7] + 2), 1), (dict(Y=P[7]), 3), (dict(Y=P[1] + 2 * 64 * 64), 3),
    (dict(Y=P[2] + 2 * 512), 3), (dict(Y=P[4] + 2 * 128), 3), (dict(G=0), 0)])
def test_grouped_w4(kw, code):
    assert grouped_w4(**kw) == code, dgt.gemm_last_error()


def loss(T=4, V=100, H=64, dtype="bf16", X=P[0], ldx=64, W=P[1], ldw=64, labels=P[2], loss=P[3], lse=P[4], ws=P[5], size=None):
    need = dgt.gemm_loss_workspace(T, V, H)
    return status("gemm_loss", (T, V, H, dtype, X, ldx, W, ldw, labels, loss, lse, ws, need if size is None else size, None))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(V=-1), 1), (dict(V=0), 1), (dict(H=-1), 1), (dict(T=1 << 31), 2), (dict(dtype="f32"), 2),
    (dict(ldx=63), 1), (dict(ldw=63), 1), (dict(X=None), 1), (dict(W=None), 1), (dict(labels=None), 1), (dict(loss=None), 1),
    (dict(labels=P[2] + 2), 1), (dict(loss=P[3] + 1), 1), (dict(lse=P[4] + 2), 1), (dict(ws=None), 1), (dict(ws=P[5] + 4), 1),
    (dict(size=100), 1), (dict(X=P[0] + 1), 1), (dict(loss=P[0]), 3), (dict(loss=P[2]), 3), (dict(lse=P[3] + 4), 3),
    (dict(lse=P[1] + 64), 3), (dict(ws=P[1]), 3), (dict(ws=P[3]), 3), (dict(ws=P[4]), 3), (dict(ws=P[2]), 3), (dict(T=0), 0),
    (dict(T=0, X=None, W=None, labels=None, loss=None, ws=None), 0)])
def test_loss(kw, code):
    assert loss(**kw) == code, dgt.gemm_last_error()


def loss_grad(T=4, V=100, H=64, dtype="bf16", X=P[0], ldx=64, W=P[1], ldw=64, labels=P[2], lse=P[3], dloss=P[4], dX=P[5],
              lddx=64, dW=P[6], lddw=64, out="f32", accumulate=0, ws=P[7], size=None):
    need = dgt.gemm_loss_grad_workspace(T, V, H)
    return status("gemm_loss_grad", (T, V, H, dtype, X, ldx, W, ldw, labels, lse, dloss, dX, lddx, dW, lddw, out, accumulate, ws,
                                     need if size is None else size, None))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(V=0), 1), (dict(H=-1), 1), (dict(V=1 << 31), 2), (dict(dtype=6), 2), (dict(out="f16"), 2),
    (dict(ldx=63), 1), (dict(ldw=63), 1), (dict(lddx=63), 1), (dict(lddw=63), 1), (dict(X=None), 1), (dict(W=None), 1),
    (dict(labels=None), 1), (dict(lse=None), 1), (dict(dloss=None), 1), (dict(ws=None), 1), (dict(ws=P[7] + 8), 1),
    (dict(size=100), 1), (dict(dX=P[5] + 1), 1), (dict(dW=P[6] + 2), 1), (dict(dX=P[0]), 3), (dict(dX=P[1]), 3),
    (dict(dW=P[1]), 3), (dict(dW=P[5]), 3), (dict(dX=P[3]), 3), (dict(dW=P[4]), 3), (dict(ws=P[5]), 3), (dict(ws=P[6]), 3),
    (dict(ws=P[0]), 3), (dict(dX=None, dW=None), 0), (dict(H=0, ldx=1, ldw=1, lddx=1, lddw=1), 0), (dict(T=0, dW=None), 0),
    (dict(T=0, accumulate=1), 0)])
def test_loss_grad(kw, code):
    assert loss_grad(**kw) == code, dgt.gemm_last_error()


def test_workspaces():
    for f, args in ((dgt.gemm_norm_grad_workspace, (100, 64)), (dgt.gemm_loss_workspace, (100, 1000, 64)),
                    (dgt.gemm_loss_grad_workspace, (100, 1000, 64))):
        assert f(*args) > 0
        assert f(-1, *args[1:]) == 0 and f(1 << 31, *args[1:]) == 0
    # Bounded by pieces of the vocabulary, not by the whole of the logits.
    assert dgt.gemm_loss_grad_workspace(8192, 1 << 20, 1024) < (1 << 30)


def test_names_raise_and_refusals_raise():
    for c in CALLS:
        with pytest.raises(KeyError):
            c.gemm_gate(0, 8, 2, "f32", None, 8, "relu", None, 1, 1, 1, 0, 1.0, None, None, None)
        with pytest.raises(KeyError):
            c.gemm_norm(0, 8, "int4", None, 8, None, None, 0.0, None, 8, None, None, None)
    with pytest.raises(TypeError):
        dgt._fast.gemm_norm(0, 8, "f32", None, 8, None, None, "small", None, 8, None, None, None)
    with pytest.raises(dgt.GemmError) as e:
        dgt.gemm_norm(4, 0, "bf16", P[0], 1, None, None, 1e-5, P[1], 1)
    assert e.value.code == dgt.GEMM_ERR_INVALID_ARG and "N=0" in str(e.value)
