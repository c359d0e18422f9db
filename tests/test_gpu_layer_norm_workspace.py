"""The layer norm gradient keeps to the workspace that it asks for, at and past
the widths where its kernels change.  Tolerances as in
test_gpu_layer_norm_many_rows.py; past 16384 columns a column sum adds at most
32 rows (of 2000) one after another in each of 64 slices."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_layer_norm import ARITH, ARITH_COLS, DT, TINY, U, ar  # noqa: E402,F401
from test_gpu_layer_norm_many_rows import make, within  # noqa: E402


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(2000, 16384), (2000, 16385), (300, 20000), (70, 50257), (500, 8193), (1500, 16383)])
def test_nothing_is_written_past_the_workspace(ar, rows, cols, dtype):
    x, dy, w, b, _ = make(rows, cols, dtype, "f32", 2, 0, 0)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ar.check(ar.ar_layer_norm(x, w, b, torch.empty_like(x), mean, rstd), "forward")
    need = ar.ar_layer_norm_workspace_bytes(rows, cols)
    around = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    ar.check(ar.ar_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, around[4096:4096 + need]), "backward")
    assert (around[:4096] == 0x5A).all() and (around[4096 + need:] == 0x5A).all()
    xh, D = (x.double() - mean.double()[:, None]) * rstd.double()[:, None], dy.double()
    for got, terms, what in ((dw, D * xh, "dweight"), (db, D, "dbias")):
        want = terms.sum(0)
        within(got, want, U["f32"] * want.abs() + ARITH_COLS * terms.abs().sum(0) + TINY["f32"], what)
    g = D * w.double()
    gx = (g * xh).mean(1, keepdim=True)
    R = rstd.double()[:, None]
    want = R * (g - g.mean(1, keepdim=True) - xh * gx)
    size = R * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    within(dx, want, U[dtype] * want.abs() + ARITH * size + TINY[dtype], "dx")
