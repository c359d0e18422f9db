"""Angles of ar_qk_norm_rope for frequencies and positions of any size.

A head of ones in the first half and zeros in the second is sqrt(2) (cos t, sin t)
for each pair.  Tolerance: sines and cosines are off by 2 units of 2^-24, the
reciprocal square root by 2, the products by 2, all of them times sqrt(2), and the
angle by 2^-33 turns, 2^-30 radians: below 10 units, 2^-20 is 16.
"""
from fractions import Fraction
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TOL = 2.0 ** -20
POSITIONS = [0, 1, -1, 3, 777, -70000, 10 ** 6, 16777217, 2 ** 31 - 1, -2 ** 31 + 1, -2 ** 31]


def two_pi(bits):
    """By Machin's formula, as a fraction that is off by 2^-bits at most."""
    one = 1 << (bits + 32)

    def arctan_of_inverse(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    return Fraction(8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)), one)


# frequencies of up to 2^1024 at positions of up to 2^31, to 2^-60 of a turn
TURN = two_pi(2300)


@pytest.fixture(scope="module")
def ar():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import binding
    torch.cuda.set_device(0)
    return binding


def check(ar, frequencies, base=10000.0, given=True):
    half = len(frequencies)
    x = torch.zeros(len(POSITIONS), 1, 2 * half, device="cuda")
    x[..., :half] = 1
    y = torch.empty_like(x)
    pos = torch.tensor(POSITIONS, dtype=torch.int32, device="cuda")
    ar.check(ar.ar_qk_norm_rope(x, None, None, None, pos, y, None, frequencies=frequencies if given else None, base=base,
                                eps=0.0), "ar_qk_norm_rope")
    turns = np.array([[float(Fraction(f) * p / TURN % 1) for f in frequencies] for p in POSITIONS])
    got = y[:, 0].double().cpu().numpy() / math.sqrt(2)
    for want, of in ((np.cos(2 * np.pi * turns), got[:, :half]), (np.sin(2 * np.pi * turns), got[:, half:])):
        off = np.abs(want - of)
        p, i = np.unravel_index(np.argmax(off), off.shape)
        assert off.max() <= TOL, (frequencies[i], POSITIONS[p], off.max())


def test_ordinary_frequencies(ar):
    check(ar, [0.0, -0.0, 1.0, -1.0, 3.7, 10.0, 0.001, 1e-7, math.pi, 2 * math.pi, -2 * math.pi, 400 * math.pi])


def test_large_frequencies(ar):
    check(ar, [1e4, 10000.1, -12345.678, 1e6, 1e8, -1e9, 2.0 ** 53 - 1, -2.0 ** 53 + 1, 1e17, 1e100, -1e200, 1e300,
               1.7976931348623157e308, -1.7976931348623157e308])


def test_small_frequencies(ar):
    check(ar, [1e-12, -1e-17, 2.0 ** -64, -2.0 ** -65, 1e-30, 1e-40, -1e-100, 2.2250738585072014e-308, 5e-324, -5e-324])


@pytest.mark.parametrize("shift", [0, 1, 17, 40, 63])
def test_frequencies_of_every_size(ar, shift):
    """Binary exponents over the whole range, so that every part of the constant counts."""
    g = np.random.Generator(np.random.PCG64(shift))
    check(ar, [float(math.ldexp(1 + g.random(), e)) for e in range(-1022 + shift, 1023, 64)])


def test_bases_below_one(ar):
    """Frequencies that grow from pair to pair, up to 1 / base."""
    for base in (1e-3, 1e-9, 0.5):
        check(ar, [base ** (-2 * i / 64) for i in range(32)], base=base, given=False)


def test_a_whole_turn_in_steps(ar):
    """Angles on both sides of every eighth of a turn, whose remainders from the
    nearest quarter have either sign: the bits of the remainder are arithmetic
    without overflow."""
    check(ar, [math.ldexp(2 * math.pi, -e) * n for e, n in ((3, 1), (3, 3), (4, 1), (5, 7), (9, 1), (9, 255), (33, 1), (33, 3))])
    steps = [2 * math.pi * (i + d) / 64 for i in range(64) for d in (-1e-7, 1e-7)]
    check(ar, steps)
    check(ar, [-f for f in steps])
