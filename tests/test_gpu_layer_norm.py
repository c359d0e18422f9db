"""ar_layer_norm and ar_layer_norm_backward against the formula in 64 bits.

Tolerances.  u is the unit roundoff of the result's type (2^-24 f32, 2^-8
bf16, 2^-11 f16): one rounding of the result costs at most u of it.  The
arithmetic before it is binary32 (unit 2^-24); a row's sums add at most 32
elements in a thread, then five levels in a warp and five across warps, so a
sum is off by at most 42 units of the sum of magnitudes, and the few products
after it add some more: 64 units, 2^-18, of the magnitudes involved.  A column
sum over at most 4096 rows adds at most 32 rows in a group, up to 16 groups of
a block and 38 + 5 levels of blocks: 128 units.
"""
import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
ARITH = 2.0 ** -18
ARITH_COLS = 2.0 ** -17


@pytest.fixture(scope="module")
def ar():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import binding
    torch.cuda.set_device(0)
    return binding


def rows_of(values, dtype, pad=0, offset=0):
    """The matrix as device rows `pad` elements apart, its first element
    `offset` elements into the allocation; the gaps hold NaN."""
    r, c = values.shape
    flat = torch.full((offset + r * (c + pad),), float("nan"), dtype=DT[dtype], device="cuda")
    m = flat[offset:].view(r, c + pad)[:, :c]
    m.copy_(torch.from_numpy(values))
    return m


def make(rows, cols, dtype, params, seed, pad=0, offset=0):
    g = np.random.Generator(np.random.PCG64(seed))
    x = rows_of(g.standard_normal((rows, cols)) * g.uniform(0.5, 2, (rows, 1)) + g.standard_normal((rows, 1)), dtype,
                pad, offset)
    dy = rows_of(g.standard_normal((rows, cols)), dtype, pad, offset)
    w = torch.from_numpy(1 + 0.2 * g.standard_normal(cols)).to("cuda", DT[params])
    b = torch.from_numpy(0.2 * g.standard_normal(cols)).to("cuda", DT[params])
    return x, dy, w, b


def f64(t):
    return t.double().cpu().numpy()


def within(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0], got[bad][:3], want[bad][:3])


def check_forward(ar, x, w, b, dtype, y, eps=1e-5):
    rows, cols = x.shape
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    X, W, B = f64(x), f64(w), f64(b) if b is not None else np.zeros(cols)
    ar.check(ar.ar_layer_norm(x, w, b, y, mean, rstd, eps=eps), "ar_layer_norm")
    m = X.mean(1, keepdims=True)
    r = 1 / np.sqrt(((X - m) ** 2).mean(1, keepdims=True) + np.float32(eps))
    want = (X - m) * r * W + B
    size = (np.abs(X) + np.abs(X).mean(1, keepdims=True)) * r
    within(f64(y), want, U[dtype] * np.abs(want) + ARITH * (size * np.abs(W) + np.abs(B)) + TINY[dtype], "y")
    within(f64(mean), m[:, 0], ARITH * np.abs(X).mean(1), "mean")
    within(f64(rstd), r[:, 0], r[:, 0] * ARITH * (1 + np.abs(X).mean(1) * r[:, 0]), "rstd")
    return mean, rstd


def check_backward(ar, dy, x, w, mean, rstd, dx, dtype, params, bias=True):
    rows, cols = x.shape
    dw = torch.full((cols,), float("nan"), dtype=DT[params], device="cuda")
    db = torch.full_like(dw, float("nan")) if bias else None
    ws = torch.full((ar.ar_layer_norm_workspace_bytes(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    DY, X, W, M, R = f64(dy), f64(x), f64(w), f64(mean)[:, None], f64(rstd)[:, None]
    ar.check(ar.ar_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws), "ar_layer_norm_backward")
    xh = (X - M) * R
    g = DY * W
    want = R * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    size = R * (np.abs(g) + np.abs(g).mean(1, keepdims=True) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    within(f64(dx), want, U[dtype] * np.abs(want) + ARITH * size + TINY[dtype], "dx")
    for got, terms, what in ((dw, DY * xh, "dweight"), (db, DY, "dbias")):
        if got is not None:
            want = terms.sum(0)
            within(f64(got), want, U[params] * np.abs(want) + ARITH_COLS * np.abs(terms).sum(0) + TINY[params], what)
    return dw, db


SHAPES = [(1, 1), (3, 5), (2, 31), (5, 32), (257, 64), (4, 96), (640, 768), (33, 771), (9, 1600), (310, 4096),
          (7, 5121), (5, 8192), (3, 8200), (2, 16384), (3, 16392), (2, 20000), (2, 40007), (4096, 40)]


@pytest.mark.parametrize("dtype,params", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                          ("f16", "f32")])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_backward(ar, rows, cols, dtype, params):
    x, dy, w, b = make(rows, cols, dtype, params, 1)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = check_forward(ar, x, w, b, dtype, y)
    check_backward(ar, dy, x, w, mean, rstd, dx, dtype, params)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 8), (5, 3)])
def test_strides_and_alignment(ar, dtype, pad, offset):
    for rows, cols in ((37, 768), (6, 1031), (3, 9000)):
        x, dy, w, b = make(rows, cols, dtype, "f32", 2, pad, offset)
        y = rows_of(np.zeros((rows, cols)), dtype, 8, 0)
        mean, rstd = check_forward(ar, x, w, b, dtype, y)
        dx = rows_of(np.zeros((rows, cols)), dtype, pad, offset)
        check_backward(ar, dy, x, w, mean, rstd, dx, dtype, "f32")
        base = y._base if y._base is not None else y
        gaps = base.flatten().view(rows, cols + 8)[:, cols:]
        assert torch.isnan(gaps).all()  # nothing is written between the rows


def test_unaligned_parameters(ar):
    x, dy, w, b = make(21, 768, "bf16", "f32", 3)
    buf = torch.zeros(2 * 768 + 3, device="cuda")
    w1, b1 = buf[1:769], buf[770:1538]
    w1.copy_(w)
    b1.copy_(b)
    y = torch.empty_like(x)
    mean, rstd = check_forward(ar, x, w1, b1, "bf16", y)
    check_backward(ar, dy, x, w1, mean, rstd, torch.empty_like(x), "bf16", "f32")


def test_in_place_without_bias_and_without_statistics(ar):
    for cols in (768, 771, 40001):
        x, dy, w, b = make(19, cols, "bf16", "bf16", 4)
        y = torch.empty_like(x)
        ar.check(ar.ar_layer_norm(x, w, None, y), "no bias")
        z = x.clone()
        mean, rstd = check_forward(ar, z.clone(), w, None, "bf16", torch.empty_like(z))
        ar.check(ar.ar_layer_norm(z, w, None, z), "in place")
        assert torch.equal(z.view(torch.int16), y.view(torch.int16))
        for which in ("dy", "x"):
            d, xx = dy.clone(), x.clone()
            dx = torch.empty_like(x)
            want = check_backward(ar, d, xx, w, mean, rstd, dx, "bf16", "bf16")
            into = d if which == "dy" else xx
            got = check_backward_bits(ar, d, xx, w, mean, rstd, into)
            assert torch.equal(into.view(torch.int16), dx.view(torch.int16))
            assert all(torch.equal(a.view(torch.int16), c.view(torch.int16)) for a, c in zip(want, got))


def check_backward_bits(ar, dy, x, w, mean, rstd, dx):
    dw, db = torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(ar.ar_layer_norm_workspace_bytes(*x.shape), dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws), "backward")
    return dw, db


def test_same_bits_every_time_and_on_another_stream(ar):
    x, dy, w, b = make(3001, 768, "f32", "f32", 5)
    y = torch.empty_like(x)
    mean, rstd = check_forward(ar, x, w, b, "f32", y)
    dx = torch.empty_like(x)
    first = [t.clone() for t in check_backward_bits(ar, dy, x, w, mean, rstd, dx)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            again = check_backward_bits(ar, dy, x, w, mean, rstd, dx)
        side.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(first, again))


def test_gradient_agrees_with_differences(ar):
    """dx, dweight and dbias against central differences of the formula's
    sum(y * dy) in 64 bits: the differences' own error is below 1e-7 of the
    magnitudes at a step of 1e-4, well below the binary32 tolerance."""
    rows, cols, eps, h = 4, 24, 1e-5, 1e-4
    x, dy, w, b = make(rows, cols, "f32", "f32", 6)
    mean, rstd = check_forward(ar, x, w, b, "f32", torch.empty_like(x))
    dx = torch.empty_like(x)
    dw, db = check_backward_bits(ar, dy, x, w, mean, rstd, dx)
    X, W, B, DY = f64(x), f64(w), f64(b), f64(dy)

    def total(X, W, B):
        m = X.mean(1, keepdims=True)
        return (((X - m) / np.sqrt(((X - m) ** 2).mean(1, keepdims=True) + eps) * W + B) * DY).sum()

    g = np.random.Generator(np.random.PCG64(7))
    for _ in range(8):
        d = [g.standard_normal(a.shape) for a in (X, W, B)]
        up = total(*(a + h * e for a, e in zip((X, W, B), d)))
        down = total(*(a - h * e for a, e in zip((X, W, B), d)))
        grads = [f64(dx), f64(dw), f64(db)]
        size = sum(np.abs(a * e).sum() for a, e in zip(grads, d))
        assert abs((up - down) / (2 * h) - sum((a * e).sum() for a, e in zip(grads, d))) <= 4e-5 * size


def test_extreme_rows(ar):
    """A constant row has variance 0: y is the bias.  A row with a NaN or an
    infinity is NaN throughout and leaves the others alone.  A row far from
    zero keeps its variance."""
    x, dy, w, b = make(6, 512, "f32", "f32", 8)
    x[0] = 3.0
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    x[3] = x[3] * 1e-2 + 1000.0
    y = torch.empty_like(x)
    mean, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    ar.check(ar.ar_layer_norm(x, w, b, y, mean, rstd), "extreme")
    assert torch.equal(y[0], b)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    for i in (3, 4, 5):
        check_forward(ar, x[i:i + 1], w, b, "f32", torch.empty_like(x[i:i + 1]))


def test_no_rows(ar):
    w = torch.ones(16, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    ar.check(ar.ar_layer_norm(x, w, w, x.clone()), "no rows")
    dw, db = torch.full((16,), 7.0, device="cuda"), torch.full((16,), 7.0, device="cuda")
    none = torch.empty(0, device="cuda")
    ar.check(ar.ar_layer_norm_backward(x, x, w, none, none, x.clone(), dw, db,
                                       torch.empty(0, device="cuda", dtype=torch.uint8)), "no rows")
    assert (dw == 0).all() and (db == 0).all()


def test_refusals(ar):
    x, dy, w, b = make(4, 64, "bf16", "f32", 9)
    y, m = torch.empty_like(x), torch.empty(4, device="cuda")
    r = torch.empty(4, device="cuda")
    bad = ar.AR_ERR_INVALID_ARG
    launches = ar.ar_kernel_launches()
    assert ar.ar_layer_norm(x, w[:63], b, y, m, r) == bad
    assert ar.ar_layer_norm(x, w, b, y[:3], m, r) == bad
    assert ar.ar_layer_norm(x, w, b, y, m[:3], r) == bad
    assert ar.ar_layer_norm(x, w, b, y, m, m) == bad                      # two outputs in one place
    assert ar.ar_layer_norm(x, w, b, y, m, r, eps=float("nan")) == bad
    assert ar.ar_layer_norm(x, w, b, y, m, r, eps=-1e-5) == bad
    assert ar.ar_layer_norm(x.t(), w, b, y.t()) == bad                    # rows are not contiguous
    assert ar.ar_layer_norm(x[:3], w, b, x[1:]) == bad                    # partly over the input
    assert ar.ar_layer_norm(x.cpu(), w, b, y) == bad                      # not device memory
    assert ar.ar_layer_norm(x, w.to(torch.float16), b.to(torch.float16), y) == ar.AR_ERR_UNSUPPORTED
    i = torch.zeros(4, 64, dtype=torch.int32, device="cuda")
    assert ar.ar_layer_norm(i, w, b, torch.empty_like(i)) == ar.AR_ERR_UNSUPPORTED
    assert ar.ar_layer_norm(x.double(), w, b, y.double()) == ar.AR_ERR_UNSUPPORTED
    assert ar.ar_layer_norm(x[:1].expand(4, 64), w, b, y) == bad          # a row stride of 0
    ws = torch.empty(ar.ar_layer_norm_workspace_bytes(4, 64), dtype=torch.uint8, device="cuda")
    dw, db = torch.empty_like(w), torch.empty_like(w)
    assert ar.ar_layer_norm_backward(dy, x, w, m, r, y, dw, db, ws[:-1]) == bad
    assert ar.ar_layer_norm_backward(dy, x, w, m, r, y, dw, dw, ws) == bad
    assert ar.ar_layer_norm_backward(dy, x, w, m, r, y, w, db, ws) == bad  # a gradient over its weight
    assert ar.ar_layer_norm_backward(dy[:, :32], x[:, :32], w[:32], m, r, x[:, 16:48], dw[:32], db[:32], ws) == bad
    assert ar.ar_kernel_launches() == launches
    # column halves of one buffer do not overlap
    wide = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, :64].copy_(x)
    ar.check(ar.ar_layer_norm(wide[:, :64], w, b, wide[:, 64:], m, r), "halves")
    ar.check(ar.ar_layer_norm(x, w, b, y, m, r), "whole")
    assert torch.equal(wide[:, 64:], y)


def test_captured_into_a_graph(ar):
    x, dy, w, b = make(65, 768, "bf16", "f32", 10)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    m, r = torch.empty(65, device="cuda"), torch.empty(65, device="cuda")
    dw, db = torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(ar.ar_layer_norm_workspace_bytes(65, 768), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ar.check(ar.ar_layer_norm(x, w, b, y, m, r), "forward")
        ar.check(ar.ar_layer_norm_backward(dy, x, w, m, r, dx, dw, db, ws), "backward")
    x.copy_(x * 1.5)
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, dx, dw, db)]
    ar.check(ar.ar_layer_norm(x, w, b, y, m, r), "forward")
    ar.check(ar.ar_layer_norm_backward(dy, x, w, m, r, dx, dw, db, ws), "backward")
    assert all(torch.equal(a, c) for a, c in itertools.zip_longest(got, (y, dx, dw, db)))


@pytest.mark.parametrize("dtype,params", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("rows,cols,pad", [(470, 9001, 0), (500, 12008, 0), (330, 16383, 5), (330, 16384, 0)])
def test_wide_rows_in_place(ar, rows, cols, pad, dtype, params):
    """Several rows to a block, so that places in shared memory are filled again."""
    x, dy, w, b = make(rows, cols, dtype, params, 60, pad)
    y = torch.empty_like(x)
    mean, rstd = check_forward(ar, x, w, b, dtype, y)
    own = rows_of(f64(x), dtype, pad)
    ar.check(ar.ar_layer_norm(own, w, b, own), "in place")
    assert torch.equal(own, y)
    want = torch.empty_like(x)
    grads = check_backward(ar, dy, x, w, mean, rstd, want, dtype, params)
    ws = torch.empty(ar.ar_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    dw, db = torch.empty_like(w), torch.empty_like(w)
    ar.check(ar.ar_layer_norm_backward(dy, x, w, mean, rstd, dy, dw, db, ws), "in place")
    assert torch.equal(dy, want) and torch.equal(dw, grads[0]) and torch.equal(db, grads[1])
    assert ar.ar_device_status() == (0, 0)
