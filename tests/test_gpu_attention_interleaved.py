"""Attention over a projection whose three parts alternate head by head,
[tokens][heads][3][dim], and its gradients written into the same layout."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_attention import ar, check, make, packed  # noqa: E402,F401


def parts(t, h, d, values=None, pad=0):
    """q, k, v as views of one [t, h, 3, d] buffer, whose rows are `pad` heads' parts longer."""
    whole = torch.full((t, h + pad, 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    views = [whole[:, :h, i] for i in range(3)]
    for view, x in zip(views, values or ()):
        view.copy_(x)
    return whole, views


@pytest.mark.parametrize("t,h,d,pad", [(333, 4, 64, 0), (200, 3, 128, 0), (140, 2, 40, 1), (1, 4, 64, 0), (130, 1, 64, 0)])
def test_three_parts_head_by_head(ar, t, h, d, pad):
    plain = make(t, h, h, d, "bf16", 90)
    dout = make(t, h, h, d, "bf16", 91)[0]
    cu = packed([t - t // 3, t // 3])
    _, (q, k, v) = parts(t, h, d, plain, pad)
    whole, grads = parts(t, h, d, pad=pad)
    out, lse, got = check(ar, q, k, v, cu, "bf16", dout, grads=grads)
    out2, lse2, want = check(ar, *plain, cu, "bf16", dout)
    assert torch.equal(out, out2) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert (whole[:, h:] == 7).all()


def test_parts_that_do_overlap_are_refused(ar):
    bad = ar.AR_ERR_INVALID_ARG
    t, h, d = 40, 4, 64
    q, k, v = make(t, h, h, d, "bf16", 92)
    out, lse, cu = torch.empty_like(q), torch.zeros(h, t, device="cuda"), packed([t])
    ws = torch.empty(ar.ar_attention_workspace_bytes(t, h, h, d), dtype=torch.uint8, device="cuda")
    whole, _ = parts(t + 1, h, d)
    flat = whole.view(-1)
    dq, dk, dv = (whole[:t, :, i] for i in range(3))

    def at(first):  # a part that begins `first` elements in
        return flat[first:].as_strided((t, h, d), (3 * h * d, 3 * d, 1))

    launches = ar.ar_kernel_launches()
    for bad_dk in (dq, at(8), at(d - 8), at(2 * d + 8), at(3 * d)):
        assert ar.ar_attention_backward(out, q, k, v, out, lse, cu, dq, bad_dk, dv, ws) == bad
    # other strides than the rest's: a head's part reaches over the next one's
    odd = flat.as_strided((t, h, d), (3 * h * d, 2 * d, 1))
    assert ar.ar_attention_backward(out, q, k, v, out, lse, cu, dq, odd[:, :, :], dv, ws) == bad
    assert ar.ar_kernel_launches() == launches
