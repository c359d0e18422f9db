"""packed_attention and diff_attention as PyTorch functions where the upstream
gradient is a part of a concatenation's and begins off a 16-byte boundary: the
gradients are those of the same numbers on one, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import distill_step
    torch.cuda.set_device(0)
    return distill_step


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("name", ["packed_attention", "diff_attention"])
def test_parts_of_a_gradient(ex, name, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    cu = torch.tensor([0, 30, 41], dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(41, n, 64, device="cuda", generator=g).to(dtype).requires_grad_() for n in (4, 4, 2))
    if name == "packed_attention":
        k = k.detach()[:, :2].contiguous().requires_grad_()
        y = ex.packed_attention(q, k, v, cu)
    else:
        y = ex.diff_attention(q, k, v, torch.full((2,), 0.5, device="cuda"), cu)
    up = torch.randn(y.numel() + 3, device="cuda", generator=g).to(dtype)
    want = torch.autograd.grad(y, (q, k, v), up[3:].clone().view_as(y), retain_graph=True)
    got = torch.autograd.grad(torch.cat((torch.zeros_like(up[:3]), y.flatten())), (q, k, v), up)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(t.abs().max() > 0 for t in want)
