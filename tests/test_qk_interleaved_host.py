"""Both directions of the norm and rotation read `interleaved` by its truth, so
that no value turns one way forward and back another.  No device is needed."""
import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("value,want", [(True, 1), (False, 0), (1, 1), (0, 0), (None, 0), (2, 1), (0.5, 1), (256, 1),
                                        (torch.tensor(True), 1)])
def test_truth(monkeypatch, value, want):
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import binding as ar
    seen = []

    class Lib:
        @staticmethod
        def ar_qk_norm_rope(*args):
            seen.append(args[14])
            return 0

        @staticmethod
        def ar_qk_norm_rope_backward(*args):
            seen.append(args[18])
            return 0

    monkeypatch.setattr(ar, "lib", Lib)
    monkeypatch.setattr(ar, "_stream_of", lambda stream, t: None)
    x, pos = torch.randn(3, 2, 8), torch.arange(3, dtype=torch.int32)
    assert ar.ar_qk_norm_rope(x, None, None, None, pos, x, None, interleaved=value) == 0
    assert ar.ar_qk_norm_rope_backward(x, None, x, None, None, None, pos, x, None, None, None, interleaved=value) == 0
    assert seen == [want, want]
