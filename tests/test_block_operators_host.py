"""Refusals of the norm and rotation, differential attention and the activation
kept in 8 bits that need no device: sizes, types, strides, alignment and
overlapping operands are judged before any CUDA call."""
import ctypes
import math

import pytest

A = 1 << 32  # addresses that are only compared
GAP = 1 << 40
F32, BF16, I32, F16 = 0, 1, 2, 3
TOO_LARGE = -6  # AR_ERR_TOO_LARGE


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


def tensor(ar, at, token=256, head=64):
    return ctypes.byref(ar.AttentionTensor(at, token, head))


# ---- norm and rotation ------------------------------------------------------------------


def turn(ar, q=None, k=None, qw=A + 2 * GAP, kw=A + 3 * GAP, positions=A + 4 * GAP, q_out=None, k_out=None, tokens=40,
         heads=4, kv=4, dim=64, rotary=64, base=10000.0, frequencies=None, eps=1e-6, dtype=BF16, wdtype=F32, none=()):
    t = {n: x or tensor(ar, A + i * GAP) for i, (n, x) in enumerate(
        (("q", q), ("k", k), ("q_out", q_out), ("k_out", k_out)), 10)}
    t.update({n: None for n in none})
    freq = None if frequencies is None else (ctypes.c_double * len(frequencies))(*frequencies)
    return ar.lib.ar_qk_norm_rope(t["q"], t["k"], qw, kw, positions, t["q_out"], t["k_out"], tokens, heads, kv, dim, rotary,
                                  base, freq, 0, eps, dtype, wdtype, None)


def test_norm_and_rotation(ar, refuses):
    bad, unsupported = ar.AR_ERR_INVALID_ARG, ar.AR_ERR_UNSUPPORTED
    assert turn(ar, tokens=-1) == bad and turn(ar, heads=0) == bad and turn(ar, kv=-1) == bad and turn(ar, dim=0) == bad
    assert turn(ar, dim=63, rotary=62) == unsupported and turn(ar, dim=258) == unsupported
    assert turn(ar, rotary=63) == bad and turn(ar, rotary=66) == bad and turn(ar, rotary=-2) == bad
    for x in (0.0, -1.0, math.nan, math.inf):
        assert turn(ar, base=x) == bad
    for x in (-1e-9, math.nan, math.inf):
        assert turn(ar, eps=x) == bad
    assert turn(ar, rotary=4, frequencies=[1.0, math.nan]) == bad
    assert turn(ar, rotary=4, frequencies=[math.inf, 1.0], base=-1.0) == bad
    assert turn(ar, dtype=9) == bad and turn(ar, wdtype=-1) == bad
    assert turn(ar, dtype=I32, wdtype=I32) == unsupported and turn(ar, dtype=F32, wdtype=BF16) == unsupported
    assert turn(ar, tokens=1 << 31) == TOO_LARGE and turn(ar, heads=(1 << 20) + 1) == TOO_LARGE
    for n in ("q", "k", "q_out", "k_out"):
        assert turn(ar, none=(n,)) == bad
    assert turn(ar, positions=None) == bad and turn(ar, positions=A + 4 * GAP + 2) == bad
    assert turn(ar, q=tensor(ar, A + 1)) == bad                               # off the element's alignment
    assert turn(ar, q=tensor(ar, A, 0)) == bad and turn(ar, k=tensor(ar, A, 256, 32)) == bad
    assert turn(ar, q=tensor(ar, A, 128, 64)) == bad                          # tokens over one another
    assert turn(ar, qw=A + 2 * GAP + 2) == bad and turn(ar, wdtype=BF16, qw=A + 2 * GAP + 1) == bad
    q = A + 10 * GAP
    assert turn(ar, q_out=tensor(ar, q + 64)) == bad                          # over q, but not in place
    assert turn(ar, q_out=tensor(ar, q, 264)) == bad                          # another stride
    assert turn(ar, q_out=tensor(ar, A + 11 * GAP)) == bad                    # in k's place
    assert turn(ar, k_out=tensor(ar, q)) == bad and turn(ar, k_out=tensor(ar, A + 12 * GAP)) == bad
    assert turn(ar, q_out=tensor(ar, A + 4 * GAP)) == bad and turn(ar, k_out=tensor(ar, A + 2 * GAP)) == bad
    assert turn(ar, tokens=0, none=("q", "k", "q_out", "k_out"), positions=None) == ar.AR_OK


def test_norm_and_rotation_backward(ar, refuses):
    bad = ar.AR_ERR_INVALID_ARG
    need = ar.ar_qk_norm_rope_workspace_bytes(40, 4, 4, 64)
    assert need > 0 and need % (64 * 4) == 0
    assert ar.ar_qk_norm_rope_workspace_bytes(-1, 4, 4, 64) == bad
    assert ar.ar_qk_norm_rope_workspace_bytes(40, 4, 4, 63) == ar.AR_ERR_UNSUPPORTED

    def back(ws=A + 20 * GAP, size=need, dq=A + 6 * GAP, dk=A + 7 * GAP, dqw=A + 8 * GAP, dkw=A + 9 * GAP, up=A):
        t = [tensor(ar, x) for x in (up, A + GAP, A + 2 * GAP, A + 3 * GAP, dq, dk)]
        return ar.lib.ar_qk_norm_rope_backward(*t[:4], A + 4 * GAP, A + 5 * GAP, A + 10 * GAP, *t[4:], dqw, dkw, 40, 4,
                                               4, 64, 64, 1e4, None, 0, 1e-6, BF16, F32, ws, size, None)
    assert back(size=need - 1) == bad and back(ws=None) == bad and back(ws=A + 20 * GAP + 2) == bad
    assert back(dk=A + 6 * GAP) == bad and back(dqw=A + 9 * GAP) == bad and back(dqw=A + 4 * GAP) == bad
    assert back(ws=A + 6 * GAP) == bad and back(up=None) == bad
    assert back(dq=A + GAP) == bad and back(dq=A + 3 * GAP) == bad            # another's upstream gradient, or input
    assert back(dq=A + 2 * GAP, dk=A + 2 * GAP) == bad


# ---- differential attention -----------------------------------------------------------------


def attend(ar, q=None, k=None, v=None, out=None, second=None, lam=A + 6 * GAP, cu=A + 7 * GAP, lse=A + 8 * GAP,
           tokens=40, seqs=2, heads=2, kv=2, dim=64, vdim=128, scale=0.125, dtype=BF16):
    t = [x or tensor(ar, A + i * GAP, 256, 128 if i > 1 else 64) for i, x in enumerate((q, k, v, out, second))]
    return ar.lib.ar_diff_attention(t[0], t[1], t[2], lam, cu, t[3], t[4], lse, tokens, seqs, heads, kv, dim, vdim,
                                    scale, dtype, None)


def test_differential_attention(ar, refuses):
    bad, unsupported = ar.AR_ERR_INVALID_ARG, ar.AR_ERR_UNSUPPORTED
    assert attend(ar, tokens=-1) == bad and attend(ar, seqs=-1) == bad and attend(ar, heads=0) == bad
    assert attend(ar, heads=3, kv=2) == bad and attend(ar, dtype=9) == bad and attend(ar, vdim=0) == bad
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert attend(ar, scale=scale) == bad
    assert attend(ar, dtype=F32) == unsupported and attend(ar, dtype=I32) == unsupported
    assert attend(ar, dim=60) == unsupported and attend(ar, dim=72) == unsupported
    assert attend(ar, vdim=60) == unsupported and attend(ar, vdim=136) == unsupported
    assert attend(ar, tokens=(1 << 30) + 1) == TOO_LARGE and attend(ar, heads=4096, kv=2) == TOO_LARGE
    assert attend(ar, tokens=1 << 29, heads=2) == TOO_LARGE
    assert attend(ar, q=tensor(ar, A + 8)) == bad                             # not on 16 bytes
    assert attend(ar, q=tensor(ar, A, 252)) == bad and attend(ar, k=tensor(ar, A + GAP, 256, 60)) == bad
    assert attend(ar, v=tensor(ar, A + 2 * GAP, 0, 128)) == bad               # every token the same row
    assert attend(ar, q=tensor(ar, A, 192, 64)) == bad                        # tokens over one another: four heads
    assert attend(ar, v=tensor(ar, A + 2 * GAP, 256, 64)) == bad              # heads over one another
    assert attend(ar, out=tensor(ar, A)) == bad and attend(ar, second=tensor(ar, A + 3 * GAP, 256, 128)) == bad
    assert attend(ar, lam=None) == bad and attend(ar, lam=A + 6 * GAP + 2) == bad
    assert attend(ar, cu=None) == bad and attend(ar, cu=A + 7 * GAP + 2) == bad
    assert attend(ar, lse=A) == bad and attend(ar, lse=A + 6 * GAP) == bad
    assert attend(ar, tokens=0) == ar.AR_OK and attend(ar, seqs=0) == ar.AR_OK


def test_differential_attention_backward(ar, refuses):
    bad = ar.AR_ERR_INVALID_ARG
    need = ar.ar_diff_attention_workspace_bytes(40, 2, 2, 64, 128)
    assert need == 40 * 4 * 4
    assert ar.ar_diff_attention_workspace_bytes(40, 3, 2, 64, 128) == bad
    assert ar.ar_diff_attention_workspace_bytes(-1, 2, 2, 64, 128) == bad
    assert ar.ar_diff_attention_workspace_bytes(40, 2, 2, 72, 128) == ar.AR_ERR_UNSUPPORTED

    def back(ws=A + 20 * GAP, size=need, lse=A + 21 * GAP, dk=A + 8 * GAP, dout=A, second=A + 5 * GAP, dlam=A + 24 * GAP,
             lam=A + 22 * GAP):
        t = [x and tensor(ar, x, 256, 128 if wide else 64) for x, wide in (
            (dout, 1), (A + GAP, 0), (A + 2 * GAP, 0), (A + 3 * GAP, 1), (A + 4 * GAP, 1), (second, 1), (A + 7 * GAP, 0),
            (dk, 0), (A + 9 * GAP, 1))]
        return ar.lib.ar_diff_attention_backward(*t[:4], lam, *t[4:6], lse, A + 23 * GAP, *t[6:], dlam, 40, 2, 2, 2, 64,
                                                 128, 0.125, BF16, ws, size, None)
    assert back(size=need - 1) == bad and back(ws=None) == bad and back(ws=A + 20 * GAP + 4) == bad
    assert back(lse=None) == bad and back(second=None) == bad and back(lam=None) == bad
    assert back(dk=A + 9 * GAP) == bad and back(dk=A + 2 * GAP) == bad and back(ws=A) == bad and back(dout=A + 4) == bad
    assert back(dlam=A + 22 * GAP) == bad and back(dlam=A + 24 * GAP + 2) == bad and back(dlam=A + 9 * GAP) == bad


# ---- activation in 8 bits -------------------------------------------------------------------


def act(ar, x=A, xs=200, y=A + GAP, ys=200, codes=A + 2 * GAP, scales=A + 3 * GAP, rows=8, cols=200, kind=1, dtype=BF16):
    return ar.lib.ar_activation8(x, xs, y, ys, codes, scales, rows, cols, kind, dtype, None)


def test_activation8(ar, refuses):
    bad = ar.AR_ERR_INVALID_ARG
    assert act(ar, rows=-1) == bad and act(ar, cols=0) == bad and act(ar, dtype=9) == bad
    assert act(ar, kind=-1) == bad and act(ar, kind=3) == bad
    assert act(ar, dtype=I32) == ar.AR_ERR_UNSUPPORTED
    assert act(ar, rows=1 << 31) == TOO_LARGE and act(ar, cols=(1 << 30) + 1, xs=1 << 31, ys=1 << 31) == TOO_LARGE
    assert act(ar, rows=(1 << 31) - 1, cols=129) == TOO_LARGE                 # blocks are counted in 31 bits
    assert act(ar, xs=199) == bad and act(ar, ys=0) == bad
    assert act(ar, x=None) == bad and act(ar, x=A + 1) == bad and act(ar, y=A + GAP + 1) == bad
    assert act(ar, codes=None) == bad and act(ar, codes=A + 2 * GAP + 8) == bad
    assert act(ar, scales=None) == bad and act(ar, scales=A + 3 * GAP + 2) == bad
    assert act(ar, y=A + 2) == bad and act(ar, y=A, ys=208) == bad            # over x, but not in place
    assert act(ar, codes=A) == bad and act(ar, scales=A + GAP) == bad and act(ar, scales=A + 2 * GAP + 8 * 256 - 4) == bad
    assert act(ar, rows=0, x=None, y=None, codes=None, scales=None) == ar.AR_OK


def test_activation8_backward(ar, refuses):
    bad = ar.AR_ERR_INVALID_ARG

    def back(codes=A, scales=A + GAP, dy=A + 2 * GAP, dys=200, dx=A + 3 * GAP, dxs=200, y=A + 4 * GAP, ys=200, rows=8,
             cols=200, kind=1, dtype=BF16):
        return ar.lib.ar_activation8_backward(codes, scales, dy, dys, dx, dxs, y, ys, rows, cols, kind, dtype, None)
    assert back(codes=None) == bad and back(codes=A + 8) == bad and back(scales=None) == bad
    assert back(dy=None) == bad and back(dx=None) == bad and back(dy=None, dx=None, y=None) == bad
    assert back(dys=100) == bad and back(dxs=100) == bad and back(ys=100) == bad
    assert back(dx=A + 2 * GAP + 4) == bad and back(y=A + 2 * GAP) == bad and back(y=A + 3 * GAP) == bad
    assert back(dx=A) == bad and back(y=A + GAP) == bad
    assert back(kind=7) == bad and back(dtype=I32) == ar.AR_ERR_UNSUPPORTED
    assert back(rows=0, codes=None, scales=None, dy=None, dx=None, y=None) == ar.AR_OK
