"""Attention backward in f16 where score gradients leave the middle of the
type's range, against the formulas in 64 bits.

Tolerances, beside those of test_gpu_attention.py (whose names they use).  A
result is rounded once: u of itself, or 2^-25, half of f16's spacing below its
smallest normal number.  What is multiplied by dout, q or k is rounded to f16
first: u of each term, or, below the type's normal numbers, half of its spacing
there.  That spacing stands for
  - 2^-40 of one for dv, as probabilities are held times 2^15,
  - 2^-25 of one for dq and dk where a block's largest score gradient lies in
    [2^-12, 65504]; below, 2^-51, as they are held times 2^26 (or 2^13 if that
    is too much for one above 2^-10); beyond, 2^-28 of the largest, as they are
    held times 2^-13 (2^-26 from 2^29 on).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_attention import U, ar, f64, make, packed, reference, within  # noqa: E402,F401

GRID = 2.0 ** -25
MOST = 60000.0  # below f16's largest number, 65504


def run(ar, q, k, v, cu, dout, scale):
    t, h, d = q.shape
    out, lse = torch.empty_like(q), torch.empty(h, t, device="cuda")
    ar.check(ar.ar_attention(q, k, v, cu, out, lse, scale=scale), "ar_attention")
    grads = [torch.full_like(x, 7.0) for x in (q, k, v)]
    ws = torch.empty(ar.ar_attention_workspace_bytes(t, h, k.shape[1], d), dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_attention_backward(dout, q, k, v, out, lse, cu, *grads, ws, scale=scale), "ar_attention_backward")
    assert ar.ar_device_status() == (0, 0)
    return out, lse, grads


def score_gradients(q, k, v, cu, scale, dout, out, lse):
    """The largest |da| of all heads."""
    most, group = 0.0, q.shape[1] // k.shape[1]
    ends = cu.tolist()
    for a, b in zip(ends, ends[1:]):
        for j in range(q.shape[1] if b > a else 0):
            g = j // group
            s = f64(q[a:b, j]) @ f64(k[a:b, g]).T * scale
            p = np.where(np.tri(b - a, dtype=bool), np.exp(s - f64(lse[j, a:b])[:, None]), 0)
            do = f64(dout[a:b, j])
            ds = p * (do @ f64(v[a:b, g]).T - (do * f64(out[a:b, j])).sum(1, keepdims=True))
            most = max(most, np.abs(ds).max())
    return most


def check(ar, q, k, v, cu, dout, scale):
    """The gradients, checked; the largest |da| and the 64-bit results."""
    out, lse, grads = run(ar, q, k, v, cu, dout, scale)
    most = score_gradients(q, k, v, cu, scale, dout, out, lse)
    r = reference(q, k, v, cu, scale, dout, out, lse)
    ds = 2.0 ** -51 if most < 2.0 ** -12 else max(2.0 ** -25, 2.0 ** -28 * most)
    lost = {"dq": ds, "dk": ds, "dv": 2.0 ** -40}
    for x, name in zip(grads, ("dq", "dk", "dv")):
        assert np.abs(r[name]).max() < MOST
        tol = U["f16"] * (np.abs(r[name]) + r[name + "_terms"]) + 2 * r[name + "_off"] + lost[name] * r[name + "_all"] + GRID
        within(f64(x), r[name], tol, name)
    return most, r


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv", [1, 4])
def test_upstream_of_a_scaled_loss(ar, dim, kv):
    """Score gradients past f16's largest number, gradients within it."""
    t = 240
    q, k, v = make(t, 4, kv, dim, "f16", 50)
    q, k = q * 0.25, k * 0.25
    v = v * 8
    dout = make(t, 4, kv, dim, "f16", 51, amplitude=4000.0 if dim == 64 else 2500.0)[0]
    most, _ = check(ar, q, k, v, packed([40, 200]), dout, 0.05)
    assert most > 1.5 * 65504


@pytest.mark.parametrize("dim", [64, 128])
def test_upstream_that_grows_along_the_sequence(ar, dim):
    """The largest score gradients are thousands of times those of the tiles
    that a block meets first."""
    t = 700
    q, k, v = make(t, 2, 1, dim, "f16", 52)
    q, k = q * 0.25, k * 0.25
    dout = make(t, 2, 1, dim, "f16", 53)[0]
    at = torch.arange(t, device="cuda")[:, None, None]
    dout = torch.where(at >= 600, dout * 8192, torch.where(at < 200, dout * 2 ** -10, dout))
    v = torch.where(at >= 400, v * 256, v)
    most, _ = check(ar, q, k, v, packed([t]), dout, 0.01)
    assert most > 65504


@pytest.mark.parametrize("dim", [64, 128])
def test_upstream_of_an_unscaled_loss(ar, dim):
    """Score gradients below what f16 can tell from zero, whose sums with large
    keys and queries are normal numbers."""
    t = 500
    q, k, v = make(t, 2, 2, dim, "f16", 54)
    dout = make(t, 2, 2, dim, "f16", 55, amplitude=2.0 ** -19)[0]
    q = q * 2.0 ** -12
    k = k * 2.0 ** 12
    most, r = check(ar, q, k, v, packed([100, 400]), dout, 2.0 ** -5)
    assert most < 2.0 ** -14 and np.abs(r["dq"]).max() > 2.0 ** -12


@pytest.mark.parametrize("dim", [64, 128])
def test_first_queries_without_a_gradient(ar, dim):
    """Upstream gradients that are zero for a sequence's first or last tokens,
    as for a prompt whose words do not count, and for all of a sequence."""
    t = 900
    q, k, v = make(t, 4, 2, dim, "f16", 56)
    dout = make(t, 4, 2, dim, "f16", 57, amplitude=2.0 ** -16)[0]
    dout[:270] = 0
    dout[420:560] = 0
    dout[600:] = 0
    check(ar, q, k, v, packed([400, 200, 300]), dout, 0.125)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("factor", [1.0, 2.0 ** -22, 30000.0])
def test_same_bits_whatever_other_sequences_hold(ar, factor, dim):
    """The power of two that score gradients are held times is each sequence's
    own affair."""
    t, lengths = 560, [130, 250, 180]
    q, k, v = make(t, 2, 1, dim, "f16", 61)
    dout = make(t, 2, 1, dim, "f16", 62)[0]
    cu = packed(lengths)
    _, _, clean = run(ar, q, k, v, cu, dout, 0.125)
    other = dout.clone()
    other[130:380] *= factor
    _, _, got = run(ar, q, k, v, cu, other, 0.125)
    for a, b in zip(clean, got):
        for at in (slice(0, 130), slice(380, 560)):
            assert torch.equal(a[at], b[at])
    _, _, again = run(ar, q, k, v, cu, other, 0.125)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, again))


@pytest.mark.parametrize("dim", [64, 128])
def test_infinite_upstream_ends(ar, dim):
    """An infinity reaches the gradients of its own sequence's tokens, those of
    keys up to 127 after its own at most; the call ends and others stay finite."""
    q, k, v = make(400, 2, 1, dim, "f16", 63)
    dout = make(400, 2, 1, dim, "f16", 64)[0]
    dout[250, 0, 3] = float("inf")
    dout[251, 1, 3] = float("nan")
    _, _, (dq, dk, dv) = run(ar, q, k, v, packed([300, 100]), dout, 0.125)
    assert not torch.isfinite(dv[0, 0, 3]) and not torch.isfinite(dq[250, 0]).all()
    for x in (dq, dk, dv):
        assert torch.isfinite(x[300:]).all()
    assert torch.isfinite(dq[:250]).all() and torch.isfinite(dk[256:]).all() and torch.isfinite(dv[256:]).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_many_blocks_call_after_call(ar, dim):
    """More blocks than the device holds, calls that nothing waits between, some
    of which walk twice: the bits of calls one by one."""
    t, heads, kv = 3000, 12, 4
    cu = packed([700, 1, 0, 1299, 514, 486])
    ws = [torch.empty(ar.ar_attention_workspace_bytes(t, heads, kv, dim), dtype=torch.uint8, device="cuda") for _ in range(3)]
    states = []
    for i, amplitude in enumerate((1.0, 2.0 ** -16, 8192.0)):
        q, k, v = make(t, heads, kv, dim, "f16", 65 + i)
        dout = make(t, heads, kv, dim, "f16", 70 + i, amplitude=amplitude)[0]
        out, lse, grads = run(ar, q, k, v, cu, dout, 0.125)
        states.append(((dout, q, k, v, out, lse, cu), grads))
    got = [[torch.full_like(x, 7.0) for x in grads] for _, grads in states]
    for n in range(60):
        i = n % 3
        ar.check(ar.ar_attention_backward(*states[i][0], *got[i], ws[i], scale=0.125), "backward")
    assert ar.ar_device_status() == (0, 0)
    for (_, want), mine in zip(states, got):
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(want, mine))
