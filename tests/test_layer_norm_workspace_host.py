"""The workspace that the layer norm gradient asks for: two floats a column for
each row of partial sums that its kernels write."""
import pytest


@pytest.fixture(scope="module")
def ar():
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import binding
    return binding


@pytest.mark.parametrize("rows,cols,partial", [
    (1, 1, 1), (5, 16384, 5), (2048, 768, 1216), (2048, 16384, 1216), (2048, 16385, 64), (2048, 50257, 64),
    (63, 50257, 63), (64, 50257, 64), (65, 50257, 64), (2 ** 31 - 1, 2 ** 30, 64), (0, 50257, 0)])
def test_partial_rows(ar, rows, cols, partial):
    """Above 16384 columns no more than 64 partial rows are written."""
    assert ar.ar_layer_norm_workspace_bytes(rows, cols) == partial * 2 * cols * 4
