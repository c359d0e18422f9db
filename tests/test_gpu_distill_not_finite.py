"""A teacher's logits that are not finite: NaN or +inf at a word of the
vocabulary make the row's distribution NaN (softmax has inf - inf there), and
so the loss and the listed words' gradients; at an entry that is no word they
do not matter."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_distill import ar, check, make  # noqa: E402,F401


@pytest.mark.parametrize("rows", [9, 1300])  # a block, or several, to a row; row after row to a block
@pytest.mark.parametrize("dtype,vdtype", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_teacher_that_is_not_finite(ar, bad, dtype, vdtype, rows):
    z, index, value, scale = make(rows, 600, 40, dtype, 70, vdtype=vdtype)
    index[:, 37] = 599  # a word, listed once
    index[:, :37] %= 599
    index[:, 38:] = -1
    loss, lse, dz = check(ar, z, index, value, scale, 2.0, dtype)
    broken = value.clone()
    broken[2, 5] = bad
    broken[3, 37] = bad
    broken[4, :] = bad
    broken[5, 38:] = bad  # no words
    broken[6, 1:38] = -float("inf")
    broken[6, 0] = bad
    broken[7, :] = -float("inf")  # no distribution: loss and gradient are zero, as documented
    rows_nan = [2, 3, 4, 6]
    l2, s2, d2, d3 = (torch.empty_like(t) for t in (loss, lse, dz, dz))
    ar.check(ar.ar_distill_loss(z, index, broken, l2, s2, scale=scale, dlogits=d2, temperature=2.0), "step")
    ar.check(ar.ar_distill_loss_backward(z, index, broken, lse, scale, d3, temperature=2.0), "backward")
    assert torch.equal(s2, lse)
    for i in range(rows):
        listed = torch.zeros(600, dtype=torch.bool, device="cuda")
        listed[index[i, :38].long()] = True
        for d in (d2, d3) if i < 12 else ():
            if i in rows_nan:
                assert torch.isnan(l2[i]) and torch.isnan(d[i, listed]).all() and torch.isfinite(d[i, ~listed]).all()
            elif i == 7:
                assert l2[i] == 0 and (d[i] == 0).all()
            else:
                assert l2[i] == loss[i] and torch.equal(d[i], dz[i])
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[rows_nan + [7]] = False
    assert torch.equal(l2[others], loss[others])
    assert torch.equal(d2[others], dz[others]) and torch.equal(d3[others], dz[others])


def test_scale_0_hides_a_broken_teacher_from_the_gradient(ar):
    """A row with scale 0 has a zero gradient, whatever it holds."""
    z, index, value, scale = make(5, 300, 6, "f32", 71)
    value[1, 2] = float("nan")
    scale[1] = 0
    loss, lse, dz = torch.empty(5, device="cuda"), torch.empty(5, device="cuda"), torch.empty_like(z)
    ar.check(ar.ar_distill_loss(z, index, value, loss, lse, scale=scale, dlogits=dz, temperature=2.0), "step")
    assert torch.isnan(loss[1]) and (dz[1] == 0).all() and torch.isfinite(dz).all()
