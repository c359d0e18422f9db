"""The PyTorch functions of a decoder block's operators in forms that the calls
below them have: queries without keys, no bias, a scale."""
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


def normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device="cuda", generator=g).to(dtype).requires_grad_()


def generator():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    return g


@pytest.mark.parametrize("weighted", [False, True])
def test_queries_without_keys(ex, weighted):
    """The same bits as with keys beside them."""
    g = generator()
    q, k, up = normal(g, 70, 4, 64), normal(g, 70, 2, 64), normal(g, 70, 4, 64).detach()
    w = normal(g, 64, dtype=torch.float32) if weighted else None
    of = [t for t in (q, w) if t is not None]
    pos = torch.arange(70, dtype=torch.int32, device="cuda")
    alone, none = ex.qk_norm_rope(q, None, w, None, pos, base=500.0)
    beside, _ = ex.qk_norm_rope(q, k, w, w, pos, base=500.0)
    assert none is None and torch.equal(alone, beside)
    got, want = torch.autograd.grad(alone, of, up), torch.autograd.grad(beside, of, up)
    assert torch.equal(got[0], want[0])
    if weighted:  # summed over as many blocks as there are queries for: 280 terms of 2^-24 in another order
        terms = (up.float() * beside.detach().float()).abs().sum((0, 1)) / w.detach().abs()
        assert ((got[1] - want[1]).abs() <= 280 * 2.0 ** -24 * 2 * terms.max()).all()


@pytest.mark.parametrize("kind", ["gelu_tanh", "gelu", "identity"])
def test_activation_without_a_bias(ex, kind):
    """A bias of zeros changes no gradient, and no result but by the rounding of
    another order of 300 products in binary32, and that to bf16."""
    g = generator()
    x, w, up = normal(g, 41, 300), normal(g, 300, 64), normal(g, 41, 64).detach()
    plain, zeros = (ex.activation8_linear(x, w, b, kind) for b in (None, torch.zeros(64, device="cuda").bfloat16()))
    size = x.detach().double().abs() @ w.detach().double().abs()
    assert ((plain - zeros).double().abs() <= 2.0 ** -8 * 2 * plain.detach().double().abs() + 300 * 2.0 ** -23 * size).all()
    got, want = (torch.autograd.grad(y, (x, w), up) for y in (plain, zeros))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(t.abs().max() > 0 for t in got)


def test_differential_attention_with_a_scale(ex):
    """A scale of 2^-3 over queries is one of 2^-2 over half of them, bit for bit,
    and its gradient twice as large: powers of two round nowhere."""
    g = generator()
    q, k, v = (normal(g, 150, n, d) for n, d in ((4, 64), (4, 64), (2, 128)))
    lam = torch.full((2,), 0.7, device="cuda").requires_grad_()
    cu, up = torch.tensor([0, 90, 150], dtype=torch.int32, device="cuda"), normal(g, 150, 2, 128).detach()
    half = (q.detach() / 2).requires_grad_()
    own = ex.diff_attention(q, k, v, lam, cu)  # dim^-1/2 = 2^-3
    given = ex.diff_attention(half, k, v, lam, cu, scale=0.25)
    assert torch.equal(own, given)
    a, b = torch.autograd.grad(own, (q, k, v, lam), up), torch.autograd.grad(given, (half, k, v, lam), up)
    assert torch.equal(2 * a[0], b[0]) and all(torch.equal(x, y) for x, y in zip(a[1:], b[1:]))
    assert not torch.equal(own, ex.diff_attention(q, k, v, lam, cu, scale=0.25))
