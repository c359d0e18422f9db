"""Attention in f16 with probabilities far below the type's smallest number,
against the formulas in 64 bits.

Tolerances, beside those of test_gpu_attention.py (whose names they use).  A
result is rounded once: u of itself, or 2^-25, half of f16's spacing below its
smallest normal number.  Probabilities are rounded to f16 for their product: u
of each term, or, below the type's normal numbers, half of its spacing there,
which stands for 2^-40 of one for dv, as they are held times 2^15, and 2^-32 of
the row's largest in the forward direction, as they are held times 2^7.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_attention import EXP, SCORE, U, ar, check, f64, make, packed, reference, within  # noqa: E402,F401

GRID = 2.0 ** -25


@pytest.mark.parametrize("dim", [64, 128])
def test_a_key_that_every_query_weighs_little(ar, dim):
    """Probabilities below 2^-25 whose sum with a large dout is a normal number."""
    t = 600
    q, k, v = make(t, 2, 2, dim, "f16", 58, amplitude=0.1)
    q[:, :, 0], k[:, :, 0] = 1, 0
    k[300, :, 0] = -12
    dout = make(t, 2, 2, dim, "f16", 59)[0] + 1000
    cu = packed([t])
    out, lse, (dq, dk, dv) = check(ar, q, k, v, cu, "f16", dout, scale=1.0)
    r = reference(q, k, v, cu, 1.0, dout, out, lse)
    assert np.abs(r["dv"][300]).min() > 2.0 ** -14
    tol = U["f16"] * (np.abs(r["dv"]) + r["dv_terms"]) + 2 * r["dv_off"] + 2.0 ** -40 * r["dv_all"] + GRID
    within(f64(dv), r["dv"], tol, "dv")


@pytest.mark.parametrize("dim", [64, 128])
def test_many_keys_that_weigh_little(ar, dim):
    """Forward: one key has nearly all the weight and a value of zero, thousands
    have 2^-26 each and large values."""
    t = 2048
    q, k, v = make(t, 1, 1, dim, "f16", 60)
    q, k = torch.zeros_like(q), torch.zeros_like(k)
    q[:, :, 0] = 1
    k[0, :, 0] = 18.0625
    v = v * 1000 + 30000
    v[0] = 0
    cu = packed([t])
    out, lse = torch.empty_like(q), torch.empty(1, t, device="cuda")
    ar.check(ar.ar_attention(q, k, v, cu, out, lse, scale=1.0), "ar_attention")
    r = reference(q, k, v, cu, 1.0)
    rel = EXP + SCORE * r["size"][..., None]
    tol = U["f16"] * np.abs(r["out"]) + (U["f16"] + rel) * r["weight"] + 2.0 ** -32 * r["all"] + GRID
    assert r["out"][-1].min() > 0.5
    within(f64(out), r["out"], tol, "out")
    within(f64(lse).T, r["lse"], SCORE * r["size"] + 2.0 ** -18 * (1 + np.abs(r["lse"])), "lse")
