"""activation8_linear as a PyTorch function without a bias: no device is needed."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def ex(monkeypatch):
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import distill_step
    kept = []

    def pack(x, y, codes, scales, kind):
        y.copy_(x * x)
        kept.append(x.detach().clone())

    def unpack(codes, scales, dy, dx, y, kind):
        y.copy_(kept[-1] ** 2)
        dx.copy_(dy * 2 * kept[-1])

    monkeypatch.setattr(distill_step, "ar", types.SimpleNamespace(
        check=lambda *a: None, ACTIVATION8_BLOCK=128, ar_activation8=pack, ar_activation8_backward=unpack))
    return distill_step


def inputs():
    g = torch.Generator()
    g.manual_seed(1)
    return [torch.randn(*s, generator=g).requires_grad_() for s in ((5, 9), (9, 4), (5, 4))]


def test_as_with_a_bias_of_zeros(ex):
    x, w, up = inputs()
    plain, zeros = ex.activation8_linear(x, w, None), ex.activation8_linear(x, w, torch.zeros(4))
    assert torch.allclose(plain, zeros, rtol=0, atol=9 * 2.0 ** -24 * (x * x).max().item() * w.abs().max().item())
    got, want = (torch.autograd.grad(y, (x, w), up.detach()) for y in (plain, zeros))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_second_derivatives_are_refused(ex):
    x, w, _ = inputs()
    grads = torch.autograd.grad(ex.activation8_linear(x, w, None).square().sum(), (x, w), create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(sum(g.square().sum() for g in grads), x)
