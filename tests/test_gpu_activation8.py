"""ar_activation8 and ar_activation8_backward against their definition: codes and
scales bit for bit, the rest in 64 bits.

Tolerances.  u is the unit roundoff of the result's type (2^-24 f32, 2^-8 bf16,
2^-11 f16), one rounding of a result.  The gelus are x times a factor whose
exponential has an argument z (z = sqrt(8/pi) (x + 0.044715 x^3), or x^2 / 2) of
binary32, off by four units of 2^-24 of itself at most, which the exponential
makes a relative error of e^-|z|, so (1 - s) times that of the factor s; its own
error, a reciprocal's (2 units each), the fitted polynomial's (4.4e-8, one unit)
and that of a few products add up to less than 32: (32 + 4 |z| (1 - s)) 2^-24 of
the value, (32 + 4 |z|) 2^-24 of the slope's other term.  What is below 2^-126 on the
way is flushed to zero, which leaves at most 2^-118 of a value or slope (times x
and u', less than 2^8 together there).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
special = pytest.importorskip("scipy.special")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -118, "bf16": 2.0 ** -118, "f16": 2.0 ** -24}
BLOCK = 128
KINDS = ("identity", "gelu_tanh", "gelu")


@pytest.fixture(scope="module")
def ar():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import binding
    torch.cuda.set_device(0)
    return binding


def f64(t):
    return t.double().cpu().numpy()


def within(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3])


def rows_of(values, dtype, pad=0, offset=0):
    """The matrix as device rows `pad` elements apart, its first element
    `offset` elements into the allocation; the gaps hold NaN."""
    r, c = values.shape
    flat = torch.full((offset + r * (c + pad),), float("nan"), dtype=DT[dtype], device="cuda")
    m = flat[offset:].view(r, c + pad)[:, :c]
    m.copy_(torch.from_numpy(values))
    return m


def like(x, fill=7.0, pad=0, offset=0):
    r, c = x.shape
    return torch.full((offset + r * (c + pad),), fill, dtype=x.dtype, device="cuda")[offset:].view(r, c + pad)[:, :c]


def kept_in_8_bits(x):
    """Codes and scales of a matrix of binary32 numbers by their definition."""
    r, c = x.shape
    full = np.zeros((r, -(-c // BLOCK) * BLOCK), np.float32)
    full[:, :c] = x
    full = full.reshape(r, -1, BLOCK)
    with np.errstate(all="ignore"):
        m = np.abs(full).max(2)
        some = (m >= np.float32(2.0 ** -120)) & np.isfinite(m)
        by = np.where(some, np.float32(127) / m, np.float32(0)).astype(np.float32)
        codes = np.where(some[..., None], np.rint(full * by[..., None]), 0).astype(np.int8)
        scales = np.where(some, m / np.float32(127), np.where(m < 2.0 ** -120, np.float32(0), np.float32(np.nan)))
    return codes.reshape(r, -1), scales.astype(np.float32)


def activation(kind, x):
    """Value, slope, and the errors of both in units of 2^-24, from the formulas."""
    if kind == "identity":
        return x, np.ones_like(x), np.abs(x), np.ones_like(x)
    if kind == "gelu":
        z, s = x * x / 2, special.ndtr(x)
        other = x * np.exp(-z) / np.sqrt(2 * np.pi)
    else:
        z = np.sqrt(8 / np.pi) * (x + 0.044715 * x ** 3)
        s = special.expit(z)
        other = x * s * special.expit(-z) * np.sqrt(8 / np.pi) * (1 + 3 * 0.044715 * x * x)
    units = 32 + 4 * np.abs(z) * (1 - s)
    return x * s, s + other, units * np.abs(x * s), units * s + (32 + 4 * np.abs(z)) * np.abs(other)


def check(ar, x, kind, dtype, dy=None, pad=0, offset=0, y=None, with_y=True, with_dx=True):
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    codes = torch.full((rows, blocks * BLOCK), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((rows, blocks), 7.0, device="cuda")
    given = f64(x)
    if y is None and with_y:
        y = like(x, 7.0, pad, offset)
    ar.check(ar.ar_activation8(x, y, codes, scales, kind=kind), "ar_activation8")
    want_codes, want_scales = kept_in_8_bits(given.astype(np.float32))
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    assert np.array_equal(scales.cpu().numpy(), want_scales, equal_nan=True)
    if y is not None:
        want, _, off, _ = activation(kind, given)
        within(f64(y), want, U[dtype] * np.abs(want) + off * 2.0 ** -24 + TINY[dtype], "y")
    if dy is None:
        return codes, scales, y
    dx = like(x, 7.0, pad, offset) if with_dx else None
    again = like(x, 7.0, pad, offset) if with_y else None
    ar.check(ar.ar_activation8_backward(codes, scales, dy if with_dx else None, dx, again, kind=kind), "ar_activation8_backward")
    xk = (want_codes.reshape(rows, blocks, BLOCK) * want_scales[..., None].astype(np.float32)).astype(np.float32)
    value, slope, voff, soff = activation(kind, xk.reshape(rows, -1)[:, :cols].astype(np.float64))
    if again is not None:
        within(f64(again), value, U[dtype] * np.abs(value) + voff * 2.0 ** -24 + TINY[dtype], "y again")
    if dx is not None:
        d = f64(dy)
        within(f64(dx), d * slope, U[dtype] * np.abs(d * slope) + np.abs(d) * (soff * 2.0 ** -24 + 2.0 ** -118)
               + TINY[dtype], "dx")
    return codes, scales, y, dx, again


def make(rows, cols, dtype, seed, pad=0, offset=0, spread=2.0):
    g = np.random.Generator(np.random.PCG64(seed))
    x = g.standard_normal((rows, cols)) * spread * np.exp(0.7 * g.standard_normal((1, cols)))
    return rows_of(x, dtype, pad, offset), rows_of(g.standard_normal((rows, cols)), dtype, pad, offset)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (2, 127), (2, 128), (4, 129), (7, 256), (3, 1000), (33, 2056)])
def test_sizes(ar, rows, cols, dtype, kind):
    x, dy = make(rows, cols, dtype, 1)
    check(ar, x, kind, dtype, dy)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 0), (8, 8), (5, 3), (1, 4)])
def test_rows_in_wider_buffers(ar, dtype, pad, offset):
    x, dy = make(9, 392, dtype, 2, pad, offset)
    check(ar, x, "gelu_tanh", dtype, dy, pad, offset)
    check(ar, x, "gelu", dtype, dy)  # the results on 16 bytes, the inputs maybe not


@pytest.mark.parametrize("dtype,cols", [("bf16", 4096), ("f32", 520), ("f16", 1001)])
def test_many_blocks(ar, dtype, cols):
    """More than a thread takes one of, the last ones short of a thread block."""
    rows = 78000 * 128 // cols + 3
    x, dy = make(rows, cols, dtype, 3)
    codes, scales, y, dx, again = check(ar, x, "gelu_tanh", dtype, dy)
    few = check(ar, x[-3:].contiguous(), "gelu_tanh", dtype, dy[-3:].contiguous())
    assert all(torch.equal(a[-3:], b) for a, b in zip((codes, scales, y, dx, again), few))


@pytest.mark.parametrize("kind", KINDS)
def test_in_place_and_parts(ar, kind):
    x, dy = make(20, 300, "bf16", 4)
    codes, scales, y, dx, again = check(ar, x, kind, "bf16", dy)
    x2, c2, s2 = x.clone(), torch.empty_like(codes), torch.empty_like(scales)
    ar.check(ar.ar_activation8(x2, x2, c2, s2, kind=kind), "in place")
    assert torch.equal(x2, y) and torch.equal(c2, codes) and torch.equal(s2, scales)
    c2.zero_()
    ar.check(ar.ar_activation8(x, None, c2, s2, kind=kind), "codes alone")
    assert torch.equal(c2, codes)
    d2 = dy.clone()
    ar.check(ar.ar_activation8_backward(codes, scales, d2, d2, None, kind=kind), "dx alone, in place")
    assert torch.equal(d2, dx)
    y2 = torch.empty_like(y)
    ar.check(ar.ar_activation8_backward(codes, scales, None, None, y2, kind=kind), "y alone")
    assert torch.equal(y2, again)


def test_ties_go_to_even_codes(ar):
    """m = 127 makes a code of each whole number; halves lie between two."""
    x = np.zeros((1, 256))
    x[0, :254] = np.arange(-126.5, 127.5, 1)
    x[0, 127] = 127
    x[0, 254] = -127
    codes, _, _ = check(ar, rows_of(x, "f32"), "identity", "f32")
    c = codes.cpu().numpy().ravel()
    assert c[0] == -126 and c[1] == -126 and c[126] == 0 and c[128] == 2 and c[254] == -127


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_small_blocks(ar, dtype):
    """Below 2^-120 a block is zeros; above, codes are as ever."""
    x = np.zeros((4, 384))
    x[0, :128] = 2.0 ** -121
    x[0, 130] = 2.0 ** -120
    x[1, :128] = np.linspace(-1, 1, 128) * 2.0 ** -119
    x[2, 300] = -2.0 ** -126
    x[3, 200] = 3e38
    x[3, 201] = -1e30
    codes, scales, _ = check(ar, rows_of(x, dtype), "gelu_tanh", dtype)
    assert (codes[0, :128] == 0).all() and codes[0, 130] == 127 and scales[2, 2] == 0 and (codes[2] == 0).all()
    d = torch.ones(4, 384, dtype=DT[dtype], device="cuda")
    dx, y = torch.empty_like(d), torch.empty_like(d)
    for kind in KINDS:
        ar.check(ar.ar_activation8_backward(codes, scales, d, dx, y, kind=kind), "backward")
        assert torch.isfinite(dx).all() and torch.isfinite(y).all()


def test_zeros(ar):
    x = torch.zeros(3, 200, device="cuda")
    for kind in KINDS:
        codes, scales, y, dx, again = check(ar, x, kind, "f32", torch.ones(3, 200, device="cuda"))
        assert (y == 0).all() and (again == 0).all() and (dx == (1 if kind == "identity" else 0.5)).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_what_is_not_finite_marks_its_block(ar, dtype, kind):
    """One NaN or infinity makes its block's gradient NaN, and no other's."""
    x, dy = make(6, 400, dtype, 5)
    clean = check(ar, x, kind, dtype, dy)
    for bad in (float("nan"), float("inf"), -float("inf")):
        x2 = x.clone()
        x2[2, 140] = bad
        codes, scales = torch.empty_like(clean[0]), torch.empty_like(clean[1])
        y, dx, again = (torch.empty_like(x) for _ in range(3))
        ar.check(ar.ar_activation8(x2, y, codes, scales, kind=kind), "forward")
        ar.check(ar.ar_activation8_backward(codes, scales, dy, dx, again, kind=kind), "backward")
        assert torch.isnan(scales[2, 1]) and (codes[2, 128:256] == 0).all()
        assert torch.isnan(dx[2, 128:256]).all() and torch.isnan(again[2, 128:256]).all()
        keep = torch.ones_like(x, dtype=torch.bool)
        keep[2, 128:256] = False
        assert torch.equal(dx[keep], clean[3][keep]) and torch.equal(again[keep], clean[4][keep])
        keep[2, 128:256] = True
        keep[2, 140] = False
        assert torch.equal(y[keep], clean[2][keep])


@pytest.mark.parametrize("kind", ["gelu_tanh", "gelu"])
def test_far_ends(ar, kind):
    """Values where an activation's factor is 0 or 1 to the last bit, and where
    its exponent leaves binary32."""
    v = np.array([-3e38, -1e20, -1e10, -100, -30, -18.5, -13.1, -10.5, -9.5, -6, -1, -1e-3, -1e-30, 0, 1e-30, 1e-3, 1, 6, 9.5,
                  10.5, 13.1, 18.5, 30, 100, 1e10, 1e20, 3e38])
    x = np.zeros((len(v), 128))
    x[:, 3] = v
    check(ar, rows_of(x, "f32"), kind, "f32", torch.ones(len(v), 128, device="cuda"))


def test_round_trip_is_within_half_a_step(ar):
    """Unpacked values are within m / 254 and roundings of what was packed."""
    x, _ = make(64, 1024, "f32", 6)
    codes, scales, _ = check(ar, x, "identity", "f32", with_y=False)
    back = torch.empty_like(x)
    ar.check(ar.ar_activation8_backward(codes, scales, None, None, back, kind="identity"), "unpack")
    m = np.abs(f64(x).reshape(64, 8, 128)).max(2, keepdims=True)
    off = np.abs(f64(back) - f64(x)).reshape(64, 8, 128)
    assert (off <= m / 254 * (1 + 2.0 ** -14)).all()


def test_gradient_agrees_with_differences(ar):
    """dx against central differences of the formula at what the codes stand
    for: at a step of 1e-3 their own error is below 1e-6 (a sixth of a third
    derivative below 3, and the value's 2^-52 over the step)."""
    x, _ = make(8, 200, "f32", 7, spread=1.0)
    dy = torch.ones_like(x)
    for kind in ("gelu_tanh", "gelu"):
        codes, scales, _, dx, _ = check(ar, x, kind, "f32", dy)
        xk = (f64(codes).reshape(8, 2, 128) * f64(scales)[..., None]).reshape(8, 256)[:, :200]
        h = 1e-3
        want = (activation(kind, xk + h)[0] - activation(kind, xk - h)[0]) / (2 * h)
        _, slope, _, soff = activation(kind, xk)
        within(f64(dx), want, 1e-6 + 2.0 ** -24 * (np.abs(slope) + soff), kind)


def test_same_bits_on_another_stream_and_in_a_graph(ar):
    x, dy = make(70, 1000, "bf16", 8)
    want = check(ar, x, "gelu", "bf16", dy)
    got = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ar.check(ar.ar_activation8(x, got[2], got[0], got[1], kind="gelu"), "forward")
        ar.check(ar.ar_activation8_backward(got[0], got[1], dy, got[3], got[4], kind="gelu"), "backward")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(ar):
    x, dy = make(10, 200, "bf16", 9)
    codes, scales = torch.empty(10, 256, dtype=torch.int8, device="cuda"), torch.empty(10, 2, device="cuda")
    y = torch.empty_like(x)
    bad, unsupported, call, back = ar.AR_ERR_INVALID_ARG, ar.AR_ERR_UNSUPPORTED, ar.ar_activation8, ar.ar_activation8_backward
    launches = ar.ar_kernel_launches()
    assert call(x.int(), y.int(), codes, scales) == unsupported and call(x.double(), None, codes, scales) == unsupported
    assert call(x, y.half(), codes, scales) == bad and call(x[0], None, codes, scales) == bad
    assert call(x, y[:9], codes, scales) == bad and call(x, y, codes[:, :200], scales) == bad
    assert call(x, y, codes.to(torch.uint8), scales) == bad and call(x, y, codes, scales.half()) == bad
    assert call(x, y, codes, scales[:, :1]) == bad and call(x, y, codes.t().contiguous().t(), scales) == bad
    assert call(x.t(), None, torch.empty(200, 128, dtype=torch.int8, device="cuda"), torch.empty(200, 1, device="cuda")) == bad
    assert call(x, y, codes.cpu(), scales) == bad
    wide = torch.empty(10, 220, dtype=torch.bfloat16, device="cuda")
    assert call(wide[:, :200], wide[:, 8:208], codes, scales) == bad
    assert back(codes, scales, dy, None, y) == bad and back(codes, scales, None, None, None) == bad
    assert back(codes, scales, dy, y, y) == bad and back(codes, scales, dy, dy, dy) == bad
    with pytest.raises(KeyError):
        call(x, y, codes, scales, kind="relu")
    assert ar.ar_kernel_launches() == launches
    none = torch.empty(0, 200, dtype=torch.bfloat16, device="cuda")
    c0, s0 = torch.empty(0, 256, dtype=torch.int8, device="cuda"), torch.empty(0, 2, device="cuda")
    assert call(none, none, c0, s0) == ar.AR_OK and back(c0, s0, none, none, none) == ar.AR_OK
    assert ar.ar_kernel_launches() == launches
