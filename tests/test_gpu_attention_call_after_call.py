"""The same call again and again, nothing waiting in between, on more blocks
than the device holds at once: the same bits every time.  Warps of a block then
run at speeds of their own, and two blocks of heads of up to 64 elements share
a multiprocessor."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_attention import DT, ar, make, packed  # noqa: E402,F401


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,heads,kv", [(64, 12, 4), (40, 12, 12), (128, 12, 4), (96, 6, 6)])
def test_same_bits_call_after_call(ar, dim, heads, kv, dtype):
    t = 3000
    cu = packed([700, 1, 0, 1299, 514, 486])
    q, k, v = make(t, heads, kv, dim, dtype, 100)
    dout = make(t, heads, kv, dim, dtype, 101)[0]
    ws = torch.empty(ar.ar_attention_workspace_bytes(t, heads, kv, dim), dtype=torch.uint8, device="cuda")

    def call(out, lse, grads, given):
        ar.check(ar.ar_attention(q, k, v, cu, out, lse), "ar_attention")
        ar.check(ar.ar_attention_backward(dout, q, k, v, *given, cu, *grads, ws), "ar_attention_backward")

    def buffers():
        return (torch.full_like(q, 7.0), torch.full((heads, t), 7.0, device="cuda"),
                [torch.full_like(x, 7.0, memory_format=torch.contiguous_format) for x in (q, k, v)])

    first = buffers()
    call(*first, first[:2])
    assert ar.ar_device_status() == (0, 0) and all(torch.isfinite(x).all() for x in (*first[:2], *first[2]))
    differ = torch.zeros(5, dtype=torch.int64, device="cuda")
    for _ in range(400):
        again = buffers()
        call(*again, first[:2])
        differ += torch.stack([(a.view(torch.int16) != b.view(torch.int16)).any().long()
                               for a, b in zip((*first[:2], *first[2]), (*again[:2], *again[2]))])
    assert differ.tolist() == [0] * 5  # calls whose out, lse, dq, dk or dv differ
    assert ar.ar_device_status() == (0, 0)
