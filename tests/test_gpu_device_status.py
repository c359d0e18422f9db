"""ar_device_status beside work of other streams."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_layer_norm import ar  # noqa: E402,F401


def test_asked_while_another_stream_is_captured(ar):
    """The status is read in the stream that is given: a capture of another
    stream goes on, and its graph holds the call made before and after."""
    x, w = torch.randn(8, 64, device="cuda"), torch.ones(64, device="cuda")
    y, z = torch.zeros_like(x), torch.zeros_like(x)
    want = torch.empty_like(x)
    ar.check(ar.ar_layer_norm(x, w, None, want), "ar_layer_norm")
    assert ar.ar_device_status() == (0, 0)
    other, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        graph.capture_begin(capture_error_mode="global")
        ar.check(ar.ar_layer_norm(x, w, None, y, stream=side), "captured")
        status = ar.ar_device_status(stream=other)
        rc = ar.ar_layer_norm(x, w, None, z, stream=side)
        graph.capture_end()
    assert status == (0, 0) and rc == ar.AR_OK
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(z, want)


def test_asked_while_a_stream_is_captured_after_a_step_wise_call(ar):
    """The same with the step-wise kernels' status word in use."""
    ranks = [torch.ones(4096, device="cuda") for _ in range(4)]
    ar.check(ar.ar_allreduce(ranks, algo="ring_stepwise"), "step-wise")
    assert ar.ar_device_status() == (0, 0)
    other, side = torch.cuda.Stream(), torch.cuda.Stream()
    y = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        graph.capture_begin(capture_error_mode="global")
        y += 1
        status = ar.ar_device_status(stream=other)
        y += 1
        graph.capture_end()
    assert status == (0, 0)
    graph.replay()
    torch.cuda.synchronize()
    assert (y == 2).all() and all((r == 4).all() for r in ranks)
