"""Attention over thousands of short sequences: what a block does to find its
own must not grow with their number."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_attention import ar, check, make, packed  # noqa: E402,F401


def lengths_of(n, seed, longest=4):
    g = np.random.Generator(np.random.PCG64(seed))
    return [int(x) for x in g.integers(0, longest, n)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("count", [255, 256, 257, 1024, 1025, 3000])
def test_thousands_of_sequences(ar, count, dim):
    """Empty ones, and some of several tiles, among them."""
    lengths = lengths_of(count, count)
    lengths[0], lengths[count // 2], lengths[-1] = 300, 700, 129
    t = sum(lengths)
    q, k, v = make(t, 2, 1, dim, "bf16", 80)
    dout = make(t, 2, 1, dim, "bf16", 81)[0]
    check(ar, q, k, v, packed(lengths), "bf16", dout)


def test_more_sequences_than_tokens_and_tokens_outside(ar):
    lengths = [0] * 5000
    lengths[17], lengths[4000], lengths[4999] = 130, 1, 40
    q, k, v = make(260, 2, 2, 64, "f16", 82)
    dout = make(260, 2, 2, 64, "f16", 83)[0]
    check(ar, q, k, v, packed(lengths, before=50), "f16", dout)
    check(ar, q, k, v, packed([0] * 3000, before=3), "f16", dout)


def test_unsound_lists_stay_inside_the_tensors(ar):
    """Entries in no order, and outside the tensors: whatever comes of it lies
    inside them, and the call ends."""
    g = np.random.Generator(np.random.PCG64(84))
    q, k, v = make(300, 2, 2, 64, "bf16", 85)
    for n in (40, 2000):
        cu = torch.from_numpy(g.integers(-100, 500, n).astype(np.int32)).cuda()
        around = torch.full((902, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        out = around[301:601]
        ar.check(ar.ar_attention(q, k, v, cu, out), "forward")
        assert ar.ar_device_status() == (0, 0)
        assert (around[:301] == 7).all() and (around[601:] == 7).all()


def test_time_grows_with_the_number_of_sequences_and_not_its_square(ar):
    """Four times as many sequences of one token: four times the blocks.  Each
    of them looking at every sequence would make it sixteen; eight lies between."""
    def took(n):
        q, k, v = make(n, 8, 8, 64, "bf16", 86)
        dout, out = torch.ones_like(q), torch.empty_like(q)
        lse, cu = torch.empty(8, n, device="cuda"), packed([1] * n)
        grads = [torch.empty_like(q) for _ in range(3)]
        ws = torch.empty(ar.ar_attention_workspace_bytes(n, 8, 8, 64), dtype=torch.uint8, device="cuda")
        best = []
        for call in (lambda: ar.ar_attention(q, k, v, cu, out, lse),
                     lambda: ar.ar_attention_backward(dout, q, k, v, out, lse, cu, *grads, ws)):
            times = []
            for _ in range(4):
                a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
                a.record()
                ar.check(call(), "call")
                b.record()
                torch.cuda.synchronize()
                times.append(a.elapsed_time(b))
            best.append(min(times))
        return best
    few, many = took(2048), took(8192)
    print("one-token sequences, ms forward and backward:", few, many)
    for a, b in zip(few, many):
        assert b <= 8 * a, (few, many)
