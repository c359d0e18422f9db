"""Attention operands of no elements are refused with a status like any other
wrong size, whether or not a scale is given."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ar():
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import binding
    return binding


@pytest.mark.parametrize("scale", [None, 0.5])
def test_heads_of_no_elements(ar, scale):
    q = torch.empty(4, 2, 0, dtype=torch.bfloat16)
    cu, lse, ws = torch.tensor([0, 4], dtype=torch.int32), torch.empty(2, 4), torch.empty(64, dtype=torch.uint8)
    bad = ar.AR_ERR_INVALID_ARG
    assert ar.ar_attention(q, q, q, cu, q, lse, scale=scale, stream=0) == bad
    assert ar.ar_attention_backward(q, q, q, q, q, lse, cu, q, q, q, ws, scale=scale, stream=0) == bad
