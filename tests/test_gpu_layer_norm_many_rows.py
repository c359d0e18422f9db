"""Layer norms with so many rows that every group of threads takes several and
its places in shared memory are filled again, against the formula in 64 bits
(on the device).

Tolerances are those of test_gpu_layer_norm.py, for the same reasons.  A column
sum there allows a group up to 32 rows: at least 152 groups have the rows of
these cases, so it is at most 32 here too (up to 4864 rows at 8192 columns,
where a multiprocessor has one group; narrower rows have more groups).
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_layer_norm import ARITH, ARITH_COLS, DT, TINY, U, ar  # noqa: E402,F401


def make(rows, cols, dtype, params, seed, pad, offset):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def matrix(values):
        flat = torch.full((offset + rows * (cols + pad),), float("nan"), dtype=DT[dtype], device="cuda")
        m = flat[offset:].view(rows, cols + pad)[:, :cols]
        m.copy_(values)
        return m

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    x = matrix(normal(rows, cols) * (torch.rand(rows, 1, device="cuda", generator=g) * 1.5 + 0.5) + normal(rows, 1))
    return (x, matrix(normal(rows, cols)), (1 + 0.2 * normal(cols)).to(DT[params]), (0.2 * normal(cols)).to(DT[params]),
            matrix)


def within(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][:3].tolist(), want[bad][:3].tolist())


CASES = [(40000, 64), (20000, 512), (20000, 768), (9000, 1600), (6000, 2048), (4500, 4096), (3000, 5120), (2500, 8192),
         (30000, 100), (15000, 771), (5000, 3001), (4000, 5121), (2500, 8191)]


@pytest.mark.parametrize("dtype,params", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"),
                                          ("f16", "f16")])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 3)])
@pytest.mark.parametrize("rows,cols", CASES)
def test_forward_and_backward(ar, rows, cols, pad, offset, dtype, params):
    x, dy, w, b, matrix = make(rows, cols, dtype, params, 1, pad, offset)
    X, W, B, DY = x.double(), w.double(), b.double(), dy.double()
    y = torch.empty(rows, cols, dtype=DT[dtype], device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ar.check(ar.ar_layer_norm(x, w, b, y, mean, rstd), "forward")
    m = X.mean(1, keepdim=True)
    r = ((X - m).square().mean(1, keepdim=True) + 1e-5) ** -0.5
    mag = X.abs().mean(1, keepdim=True)
    want = (X - m) * r * W + B
    within(y, want, U[dtype] * want.abs() + ARITH * ((X.abs() + mag) * r * W.abs() + B.abs()) + TINY[dtype], "y")
    within(mean, m[:, 0], ARITH * mag[:, 0], "mean")
    within(rstd, r[:, 0], r[:, 0] * ARITH * (1 + mag[:, 0] * r[:, 0]), "rstd")
    own = matrix(x)
    ar.check(ar.ar_layer_norm(own, w, b, own), "in place")
    assert torch.equal(own, y)

    dx = torch.empty(rows, cols, dtype=DT[dtype], device="cuda")
    dw, db = (torch.full((cols,), float("nan"), dtype=DT[params], device="cuda") for _ in range(2))
    ws = torch.full((ar.ar_layer_norm_workspace_bytes(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws), "backward")
    M, R = mean.double()[:, None], rstd.double()[:, None]
    xh, g = (X - M) * R, DY * W
    gx = (g * xh).mean(1, keepdim=True)
    want = R * (g - g.mean(1, keepdim=True) - xh * gx)
    size = R * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    within(dx, want, U[dtype] * want.abs() + ARITH * size + TINY[dtype], "dx")
    for got, terms, what in ((dw, DY * xh, "dweight"), (db, DY, "dbias")):
        want = terms.sum(0)
        within(got, want, U[params] * want.abs() + ARITH_COLS * terms.abs().sum(0) + TINY[params], what)
    kept = dx.clone()
    dw2 = torch.empty_like(dw)
    ar.check(ar.ar_layer_norm_backward(dy, x, w, mean, rstd, dy, dw2, None, ws), "in place, without dbias")
    assert torch.equal(dy, kept) and torch.equal(dw2, dw)
    assert ar.ar_device_status() == (0, 0)
