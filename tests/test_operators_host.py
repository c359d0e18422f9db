"""The training-step operators' refusals that need no device: sizes, types,
strides, alignment and overlapping operands are judged before any CUDA call."""
import ctypes
import math

import pytest

A = 1 << 32  # addresses that are only compared
GAP = 1 << 40


@pytest.fixture(scope="module")
def ar():
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import binding
    return binding


@pytest.fixture
def refuses(ar):
    launches = ar.ar_kernel_launches()
    yield
    assert ar.ar_kernel_launches() == launches


F32, BF16, I32, F16 = 0, 1, 2, 3
TOO_LARGE = -6  # AR_ERR_TOO_LARGE


def norm(ar, x=A, xs=64, w=A + GAP, b=A + 2 * GAP, y=A + 3 * GAP, ys=64, mean=A + 4 * GAP, rstd=A + 5 * GAP, rows=8,
         cols=64, eps=1e-5, dtype=BF16, pdtype=F32):
    return ar.lib.ar_layer_norm(x, xs, w, b, y, ys, mean, rstd, rows, cols, eps, dtype, pdtype, None)


def test_layer_norm(ar, refuses):
    bad = ar.AR_ERR_INVALID_ARG
    assert norm(ar, rows=-1) == bad and norm(ar, cols=0) == bad and norm(ar, dtype=9) == bad
    assert norm(ar, dtype=I32, pdtype=I32) == ar.AR_ERR_UNSUPPORTED
    assert norm(ar, dtype=F32, pdtype=BF16) == ar.AR_ERR_UNSUPPORTED
    assert norm(ar, dtype=F16, pdtype=BF16) == ar.AR_ERR_UNSUPPORTED
    assert norm(ar, rows=1 << 31) == TOO_LARGE
    assert norm(ar, cols=(1 << 30) + 1, xs=1 << 31, ys=1 << 31) == TOO_LARGE
    for eps in (-1e-9, math.nan, math.inf):
        assert norm(ar, eps=eps) == bad
    assert norm(ar, xs=63) == bad and norm(ar, ys=0) == bad
    assert norm(ar, x=None) == bad and norm(ar, w=None) == bad and norm(ar, y=None) == bad
    assert norm(ar, x=A + 1) == bad and norm(ar, w=A + GAP + 2) == bad and norm(ar, mean=A + 4 * GAP + 2) == bad
    assert norm(ar, y=A + 2) == bad and norm(ar, y=A, ys=65, xs=64) == bad      # overlaps, not in place
    assert norm(ar, mean=A) == bad and norm(ar, rstd=A + 4 * GAP) == bad and norm(ar, y=A + GAP) == bad
    assert norm(ar, rows=0, x=None, w=None, y=None) == ar.AR_OK


def norm_back(ar, dy=A, x=A + GAP, w=A + 2 * GAP, mean=A + 3 * GAP, rstd=A + 4 * GAP, dx=A + 5 * GAP, dw=A + 6 * GAP,
              db=A + 7 * GAP, rows=8, cols=64, stride=64, ws=A + 8 * GAP, size=1 << 30):
    return ar.lib.ar_layer_norm_backward(dy, stride, x, stride, w, mean, rstd, dx, stride, dw, db, rows, cols, BF16,
                                         F32, ws, size, None)


def test_layer_norm_backward(ar, refuses):
    bad = ar.AR_ERR_INVALID_ARG
    need = ar.ar_layer_norm_workspace_bytes(8, 64)
    assert need == 8 * 2 * 64 * 4
    assert norm_back(ar, size=need - 1) == bad and norm_back(ar, ws=None, size=need) == bad
    assert norm_back(ar, ws=A + 8 * GAP + 2) == bad
    assert norm_back(ar, mean=None) == bad and norm_back(ar, dw=None) == bad and norm_back(ar, dx=None) == bad
    assert norm_back(ar, dw=A + 7 * GAP) == bad and norm_back(ar, dw=A) == bad and norm_back(ar, dx=A + 64) == bad
    assert norm_back(ar, stride=60) == bad
    assert ar.ar_layer_norm_workspace_bytes(-1, 8) == bad and ar.ar_layer_norm_workspace_bytes(8, 0) == bad
    assert ar.ar_layer_norm_workspace_bytes(1 << 20, 768) == 1216 * 2 * 768 * 4


def distill(ar, z=A, zs=100, index=A + GAP, value=A + 2 * GAP, scale=None, loss=A + 3 * GAP, lse=A + 4 * GAP,
            dz=A + 5 * GAP, ds=100, rows=8, vocab=100, top=4, tau=1.0, dtype=BF16, vdtype=F32):
    return ar.lib.ar_distill_loss(z, zs, index, value, scale, loss, lse, dz, ds, rows, vocab, top, tau, dtype, vdtype,
                                  None)


def test_distill(ar, refuses):
    bad = ar.AR_ERR_INVALID_ARG
    for tau in (0.0, -1.0, math.nan, math.inf):
        assert distill(ar, tau=tau) == bad
    assert distill(ar, rows=-1) == bad and distill(ar, vocab=0) == bad and distill(ar, top=-1) == bad
    assert distill(ar, dtype=I32) == ar.AR_ERR_UNSUPPORTED and distill(ar, vdtype=F16) == ar.AR_ERR_UNSUPPORTED
    assert distill(ar, top=1025) == TOO_LARGE
    assert distill(ar, vocab=(1 << 30) + 1, zs=1 << 31, ds=1 << 31) == TOO_LARGE
    assert distill(ar, zs=99) == bad and distill(ar, ds=99) == bad
    assert distill(ar, z=None) == bad and distill(ar, index=None) == bad and distill(ar, loss=None) == bad
    assert distill(ar, dz=A + 2) == bad and distill(ar, dz=A, ds=104) == bad and distill(ar, loss=A + 4 * GAP) == bad
    assert distill(ar, lse=A) == bad and distill(ar, scale=A + 3 * GAP) == bad
    assert distill(ar, rows=0, z=None) == ar.AR_OK
    assert ar.lib.ar_distill_loss_backward(A, 100, A + GAP, A + 2 * GAP, A + 3 * GAP, None, A + 5 * GAP, 100, 8, 100, 4,
                                           1.0, BF16, F32, None) == bad
    assert ar.lib.ar_distill_loss_backward(A, 100, A + GAP, A + 2 * GAP, A + 3 * GAP, A + 4 * GAP, None, 100, 8, 100, 4,
                                           1.0, BF16, F32, None) == bad


def tensor(ar, at, token=256, head=64):
    return ctypes.byref(ar.AttentionTensor(at, token, head))


def attend(ar, q=None, k=None, v=None, out=None, cu=A + 4 * GAP, lse=A + 5 * GAP, tokens=40, seqs=2, heads=4, kv=4,
           dim=64, scale=0.125, dtype=BF16):
    t = [x or tensor(ar, A + i * GAP) for i, x in enumerate((q, k, v, out))]
    return ar.lib.ar_attention(t[0], t[1], t[2], cu, t[3], lse, tokens, seqs, heads, kv, dim, scale, dtype, None)


def test_attention(ar, refuses):
    bad, unsupported = ar.AR_ERR_INVALID_ARG, ar.AR_ERR_UNSUPPORTED
    assert attend(ar, tokens=-1) == bad and attend(ar, seqs=-1) == bad and attend(ar, heads=0) == bad
    assert attend(ar, heads=3, kv=2) == bad and attend(ar, dtype=9) == bad
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert attend(ar, scale=scale) == bad
    assert attend(ar, dtype=F32) == unsupported and attend(ar, dtype=I32) == unsupported
    assert attend(ar, dim=60) == unsupported and attend(ar, dim=136) == unsupported
    assert attend(ar, tokens=(1 << 30) + 1) == TOO_LARGE and attend(ar, heads=8192) == TOO_LARGE
    assert attend(ar, tokens=1 << 30, heads=4) == TOO_LARGE
    assert attend(ar, q=tensor(ar, A + 8)) == bad                           # not on 16 bytes
    assert attend(ar, q=tensor(ar, A, 252)) == bad and attend(ar, k=tensor(ar, A + GAP, 256, 60)) == bad
    assert attend(ar, v=tensor(ar, A + 2 * GAP, 0)) == bad                  # every token the same row
    assert attend(ar, q=tensor(ar, A, 128, 64)) == bad                      # tokens over one another
    assert attend(ar, out=tensor(ar, A)) == bad and attend(ar, out=tensor(ar, A + 2 * GAP + 64)) == bad
    assert attend(ar, cu=None) == bad and attend(ar, cu=A + 4 * GAP + 2) == bad and attend(ar, lse=A) == bad
    assert attend(ar, tokens=0) == ar.AR_OK and attend(ar, seqs=0) == ar.AR_OK


def test_attention_backward(ar, refuses):
    bad = ar.AR_ERR_INVALID_ARG
    need = ar.ar_attention_workspace_bytes(40, 4, 2, 64)
    assert need == 40 * 4 * 4
    assert ar.ar_attention_workspace_bytes(40, 3, 2, 64) == bad
    assert ar.ar_attention_workspace_bytes(-1, 4, 2, 64) == bad
    assert ar.ar_attention_workspace_bytes(40, 4, 2, 63) == ar.AR_ERR_UNSUPPORTED

    def back(ws=A + 20 * GAP, size=need, lse=A + 21 * GAP, dk=A + 7 * GAP, dout=A):
        t = [tensor(ar, x, 128 if kv else 256) for x, kv in (
            (dout, 0), (A + GAP, 0), (A + 2 * GAP, 1), (A + 3 * GAP, 1), (A + 4 * GAP, 0), (A + 6 * GAP, 0), (dk, 1),
            (A + 8 * GAP, 1))]
        return ar.lib.ar_attention_backward(*t[:5], lse, A + 22 * GAP, *t[5:], 40, 2, 4, 2, 64, 0.125, BF16, ws, size,
                                            None)
    assert back(size=need - 1) == bad and back(ws=None) == bad and back(ws=A + 20 * GAP + 4) == bad
    assert back(lse=None) == bad and back(dk=A + 8 * GAP) == bad and back(dk=A + 2 * GAP) == bad
    assert back(ws=A) == bad and back(dout=A + 4) == bad
