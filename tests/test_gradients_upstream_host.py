"""packed_attention and diff_attention as PyTorch functions where the upstream
gradient is a part of a larger one and begins off a 16-byte boundary, which the
calls refuse: they are given it on one.  No device is needed."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def ex(monkeypatch):
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import distill_step

    def attention(q, k, v, *rest, **how):
        out = rest[-2] if len(rest) == 3 else rest[2]
        out.copy_(v.repeat(1, out.shape[1] // v.shape[1], 1))

    def backward(dout, q, k, v, *rest, **how):
        # the calls' own conditions for an operand
        assert dout.data_ptr() % 16 == 0 and dout.stride() == (dout.shape[1] * dout.shape[2], dout.shape[2], 1)
        seen.append(dout.clone())

    seen = []
    fake = types.SimpleNamespace(check=lambda *a: None, ar_attention=attention, ar_attention_backward=backward,
                                 ar_attention_workspace_bytes=lambda *a: 16, ar_diff_attention=attention,
                                 ar_diff_attention_backward=backward, ar_diff_attention_workspace_bytes=lambda *a: 16)
    monkeypatch.setattr(distill_step, "ar", fake)
    return distill_step, seen


@pytest.mark.parametrize("skipped", [0, 1, 3, 4])
@pytest.mark.parametrize("name", ["packed_attention", "diff_attention"])
def test_parts_of_a_gradient(ex, name, skipped):
    f, seen = ex
    cu = torch.tensor([0, 5], dtype=torch.int32)
    g = torch.Generator()
    g.manual_seed(1)
    heads = (2, 2, 2) if name == "packed_attention" else (4, 4, 2)
    q, k, v = (torch.randn(5, n, 8, generator=g).requires_grad_() for n in heads)
    y = f.packed_attention(q, k, v, cu) if name == "packed_attention" else f.diff_attention(q, k, v, torch.ones(2), cu)
    up = torch.randn(skipped + y.numel(), generator=g)
    torch.autograd.grad(torch.cat((torch.zeros(skipped), y.flatten())), (q, k, v), up)
    assert torch.equal(seen[0].flatten(), up[skipped:])
