"""layer_norm as a PyTorch function with and without a bias, on the device."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_distill_step import ex  # noqa: E402,F401


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_without_bias_are_those_of_a_bias_of_zero(ex, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, dy = (torch.randn(300, 768, device="cuda", generator=g).to(dtype) for _ in range(2))
    w = torch.randn(768, device="cuda", generator=g)
    results = []
    for bias in (None, torch.zeros(768, device="cuda")):
        a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
        y = ex.layer_norm(a, b, bias)
        y.backward(dy)
        results.append((y.detach(), a.grad, b.grad))
    assert all(torch.equal(p, q) for p, q in zip(*results))
