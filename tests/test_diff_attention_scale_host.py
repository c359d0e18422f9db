"""diff_attention as a PyTorch function with a scale of the caller's, which both
directions get; without one both take the calls' own.  No device is needed."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("how", [{}, {"scale": 0.5}, {"scale": None}])
def test_scale_reaches_both_calls(monkeypatch, how):
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import distill_step
    seen = []

    def call(*operands, scale=None):
        seen.append(scale)

    monkeypatch.setattr(distill_step, "ar", types.SimpleNamespace(
        check=lambda *a: None, ar_diff_attention=call, ar_diff_attention_backward=call,
        ar_diff_attention_workspace_bytes=lambda *a: 16))
    q, k, v = (torch.randn(5, n, 8).requires_grad_() for n in (4, 4, 2))
    y = distill_step.diff_attention(q, k, v, torch.ones(2), torch.tensor([0, 5], dtype=torch.int32), **how)
    y.sum().backward()
    assert seen == [how.get("scale")] * 2
