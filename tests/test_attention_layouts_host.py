"""Which arrangements of attention operands share bytes, against the sets of
their addresses.  Sharing is judged before any CUDA call: what shares a byte is
AR_ERR_INVALID_ARG, and what does not gets as far as the device, of which there
is none here."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

BASE, FAR = 1 << 40, 1 << 44


@pytest.fixture(scope="module")
def ar():
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import binding
    return binding


def call(ar, q, out, tokens, heads, dim):
    """ar_attention with q and out as (address, token stride, head stride), the rest far away."""
    t = [ctypes.byref(ar.AttentionTensor(*x)) for x in (q, (FAR, heads * dim, dim), (2 * FAR, heads * dim, dim), out)]
    return ar.lib.ar_attention(t[0], t[1], t[2], 3 * FAR, t[3], None, tokens, 2, heads, heads, dim, 0.125, 1, None)


def elements(x, tokens, heads, dim):
    at, ts, hs = x
    return {at // 2 + t * ts + h * hs + i for t in range(tokens) for h in range(heads) for i in range(0, dim, 8)}


def arrangement(g, tokens, heads, dim):
    hs = dim * int(g.integers(1, 4)) + 8 * int(g.integers(0, 2))
    if g.random() < 0.5:
        return hs * (heads + int(g.integers(0, 2))) + 8 * int(g.integers(0, 3)), hs  # tokens outside
    return hs, hs * (tokens + int(g.integers(0, 2)))                                # heads outside


def test_nothing_that_shares_a_byte_is_accepted(ar):
    g = np.random.Generator(np.random.PCG64(1))
    shared = apart = 0
    for _ in range(4000):
        tokens, heads, dim = int(g.integers(1, 5)), int(g.integers(1, 5)), int(g.choice([8, 16, 24]))
        s = arrangement(g, tokens, heads, dim)
        r = s if g.random() < 0.6 else arrangement(g, tokens, heads, dim)
        q = (BASE, *s)
        out = (BASE + 16 * int(g.integers(-12, 12)), *r)
        same = elements(q, tokens, heads, dim) & elements(out, tokens, heads, dim)
        rc = call(ar, q, out, tokens, heads, dim)
        if same:
            shared += 1
            assert rc == ar.AR_ERR_INVALID_ARG, (q, out, tokens, heads, dim)
        else:
            apart += 1
    assert shared > 500 and apart > 500


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no device memory, which is the same status")
@pytest.mark.parametrize("tokens,heads,dim,pad", [(5, 4, 64, 0), (1, 3, 8, 0), (7, 1, 16, 0), (3, 2, 40, 1), (4, 5, 128, 0)])
def test_parts_head_by_head_are_accepted(ar, tokens, heads, dim, pad):
    s = ((heads + pad) * 3 * dim, 3 * dim)
    for a in range(3):
        for b in range(3):
            rc = call(ar, (BASE + 2 * a * dim, *s), (BASE + 2 * b * dim, *s), tokens, heads, dim)
            assert (rc == ar.AR_ERR_INVALID_ARG) == (a == b)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no device memory, which is the same status")
def test_tokens_of_alternating_buffers_are_accepted(ar):
    """Heads outside, and the tokens of two buffers by turns within a head."""
    tokens, heads, dim = 6, 3, 32
    s = (2 * dim, 2 * dim * tokens)
    assert call(ar, (BASE, *s), (BASE + 2 * dim, *s), tokens, heads, dim) != ar.AR_ERR_INVALID_ARG
    assert call(ar, (BASE, *s), (BASE + 2 * dim - 16, *s), tokens, heads, dim) == ar.AR_ERR_INVALID_ARG
