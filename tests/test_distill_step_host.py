"""The PyTorch functions of distill_step with the library's calls replaced by
their formulas: no device is needed."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def ex(monkeypatch):
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import distill_step

    def norm(x, weight, bias, y, mean, rstd, eps):
        mean.copy_(x.mean(1))
        rstd.copy_((x.var(1, correction=0) + eps).rsqrt())
        y.copy_((x - mean[:, None]) * rstd[:, None] * weight + (0 if bias is None else bias))

    def norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace):
        xh, g = (x - mean[:, None]) * rstd[:, None], dy * weight
        dx.copy_(rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)))
        dweight.copy_((dy * xh).sum(0))
        if dbias is not None:
            dbias.copy_(dy.sum(0))

    def scores(q, k, lse=None):  # one sequence, as many heads of k as of q
        s = torch.einsum("ihd,jhd->hij", q, k) * q.shape[2] ** -0.5
        return s.masked_fill(torch.ones(len(q), len(q), dtype=torch.bool).triu(1), -float("inf"))

    def attention(q, k, v, cu_seqlens, out, lse):
        s = scores(q, k)
        lse.copy_(s.logsumexp(2))
        out.copy_(torch.einsum("hij,jhd->ihd", s.softmax(2), v))

    def attention_backward(dout, q, k, v, out, lse, cu_seqlens, dq, dk, dv, workspace):
        p = (scores(q, k) - lse[:, :, None]).exp()
        dp = torch.einsum("ihd,jhd->hij", dout, v)
        ds = p * (dp - (dout * out).sum(2).t()[:, :, None]) * q.shape[2] ** -0.5
        dq.copy_(torch.einsum("hij,jhd->ihd", ds, k))
        dk.copy_(torch.einsum("hij,ihd->jhd", ds, q))
        dv.copy_(torch.einsum("hij,ihd->jhd", p, dout))

    def loss(logits, index, value, out, lse, temperature):
        lse.copy_((logits / temperature).logsumexp(1))
        p = (value / temperature).softmax(1)
        out.copy_(temperature ** 2 * (p * (p.log() - logits.gather(1, index.long()) / temperature + lse[:, None])).sum(1))

    def loss_backward(logits, index, value, lse, dloss, dlogits, temperature):
        q = (logits / temperature - lse[:, None]).exp()
        p = (value / temperature).softmax(1)
        dlogits.copy_(q.scatter_add(1, index.long(), -p) * (dloss * temperature)[:, None])

    monkeypatch.setattr(distill_step, "ar", types.SimpleNamespace(
        check=lambda *a: None, ar_layer_norm=norm, ar_layer_norm_backward=norm_backward,
        ar_layer_norm_workspace_bytes=lambda *a: 16, ar_attention=attention, ar_attention_backward=attention_backward,
        ar_attention_workspace_bytes=lambda *a: 16, ar_distill_loss=loss, ar_distill_loss_backward=loss_backward))
    return distill_step


def cases(ex):
    g = torch.Generator()
    g.manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g).requires_grad_()

    index = torch.randint(9, (5, 3), generator=g, dtype=torch.int32)
    cu = torch.tensor([0, 6], dtype=torch.int32)
    return {"layer_norm": (ex.layer_norm, (normal(5, 8), normal(8), normal(8))),
            "layer_norm without bias": (lambda x, w: ex.layer_norm(x, w, None), (normal(5, 8), normal(8))),
            "packed_attention": (lambda q, k, v: ex.packed_attention(q, k, v, cu), tuple(normal(6, 2, 8) for _ in range(3))),
            "distill_loss": (lambda z: ex.distill_loss(z, index, torch.zeros(5, 3), 2.0), (normal(5, 9),))}


NAMES = ["layer_norm", "packed_attention", "distill_loss"]


@pytest.mark.parametrize("name", NAMES + ["layer_norm without bias"])
def test_first_derivatives(ex, name):
    """Against differences of the replaced calls in 32 bits: off by 1e-3 of the
    magnitudes at a step of 1e-2 (its cube's third and binary32's rounding)."""
    f, inputs = cases(ex)[name]
    y = f(*inputs)
    g = torch.Generator()
    g.manual_seed(2)
    up = torch.randn(y.shape, generator=g)
    grads = torch.autograd.grad(y, inputs, up)
    h = 1e-2
    d = [torch.randn(x.shape, generator=g) for x in inputs]
    with torch.no_grad():
        plus, minus = (f(*(x + s * h * e for x, e in zip(inputs, d))) for s in (1, -1))
    want = ((plus.double() - minus.double()) * up / (2 * h)).sum()
    got = sum((a * e).sum() for a, e in zip(grads, d))
    size = sum((a * e).abs().sum() for a, e in zip(grads, d))
    assert abs(want - got) <= 1e-3 * size


@pytest.mark.parametrize("name", NAMES)
def test_second_derivatives_are_refused(ex, name):
    """The gradients are not differentiable themselves: asking for it raises,
    and is not answered as if they were constants."""
    f, inputs = cases(ex)[name]
    loss = f(*inputs).square().sum()
    grads = torch.autograd.grad(loss, inputs, create_graph=True)
    penalty = sum(g.square().sum() for g in grads) + sum(x.square().sum() for x in inputs)
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(penalty, inputs, retain_graph=True)
    for x in inputs:  # each by itself
        with pytest.raises(RuntimeError, match="second derivatives"):
            torch.autograd.grad(penalty, x, retain_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        penalty.backward()


@pytest.mark.parametrize("name", NAMES)
def test_a_graph_of_the_gradients_alone_changes_nothing(ex, name):
    f, inputs = cases(ex)[name]
    y = f(*inputs)
    plain = torch.autograd.grad(y.sum(), inputs, retain_graph=True)
    graphed = torch.autograd.grad(y.sum(), inputs, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, graphed))
    y.sum().backward()
    assert all(torch.equal(x.grad, a) for x, a in zip(inputs, plain))
