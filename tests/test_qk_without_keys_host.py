"""qk_norm_rope as a PyTorch function of queries alone, as the calls below it
allow: no device is needed."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def ex(monkeypatch):
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import distill_step

    def forward(q, k, q_weight, k_weight, positions, q_out, k_out, **how):
        assert (k is None) == (k_out is None)
        q_out.copy_(q * q_weight)
        if k is not None:
            k_out.copy_(k * k_weight)

    def backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, dq, dk, dq_weight, dk_weight, workspace, **how):
        assert (k is None) == (dk_out is None) == (dk is None)
        dq.copy_(dq_out * q_weight)
        dq_weight.copy_((dq_out * q).sum((0, 1)))
        if k is not None:
            dk.copy_(dk_out * k_weight)
            dk_weight.copy_((dk_out * k).sum((0, 1)))
        elif dk_weight is not None:
            dk_weight.zero_()

    def workspace_bytes(tokens, heads, kv_heads, dim):
        assert (tokens, heads, dim) == (5, 3, 8) and kv_heads in (0, 2)
        return 16

    monkeypatch.setattr(distill_step, "ar", types.SimpleNamespace(
        check=lambda *a: None, ar_qk_norm_rope=forward, ar_qk_norm_rope_backward=backward,
        ar_qk_norm_rope_workspace_bytes=workspace_bytes))
    return distill_step


def inputs():
    g = torch.Generator()
    g.manual_seed(1)
    q, k, a, b = (torch.randn(*s, generator=g).requires_grad_() for s in ((5, 3, 8), (5, 2, 8), (8,), (8,)))
    return q, k, a, b, torch.arange(5, dtype=torch.int32)


def test_queries_alone(ex):
    q, k, a, b, pos = inputs()
    q_out, k_out = ex.qk_norm_rope(q, None, a, None, pos)
    with_keys, _ = ex.qk_norm_rope(q, k, a, b, pos)
    assert k_out is None and torch.equal(q_out, with_keys)
    up = torch.randn(q.shape)
    got, want = (torch.autograd.grad(y, (q, a), up) for y in (q_out, with_keys))
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_weight_of_no_keys_has_a_zero_gradient(ex):
    q, _, a, b, pos = inputs()
    q_out, _ = ex.qk_norm_rope(q, None, a, b, pos)
    dq, db = torch.autograd.grad(q_out.sum(), (q, b))
    assert (db == 0).all() and torch.equal(dq, a.expand_as(dq))


def test_second_derivatives_are_refused(ex):
    q, _, a, _, pos = inputs()
    q_out, _ = ex.qk_norm_rope(q, None, a, None, pos)
    grads = torch.autograd.grad(q_out.square().sum(), (q, a), create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(sum(g.square().sum() for g in grads), q)
