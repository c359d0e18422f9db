"""The operators together, in the example's data-parallel training step."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import distill_step
    torch.cuda.set_device(0)
    return distill_step


def plain_norm(x, weight, bias):
    return torch.nn.functional.layer_norm(x, x.shape[1:], weight, bias)


def plain_attention(q, k, v, cu_seqlens):
    c = cu_seqlens.tolist()
    parts = []
    for a, b in zip(c, c[1:]):
        s = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b]) * q.shape[2] ** -0.5
        s = s.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool).triu(1), -float("inf"))
        parts.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), v[a:b]))
    return torch.cat(parts)


def plain_loss(z, b, temperature):
    p = (b["teacher_logits"].double() / temperature).softmax(1)
    q = (z / temperature).log_softmax(1).gather(1, b["teacher_index"].long())
    return temperature ** 2 * (p * (p.log() - q)).sum(1).mean()


def test_gradients_of_the_whole_model(ex):
    """Against the same model in 64 bits on the CPU.  An activation or a
    gradient is rounded to bf16 some forty times on its way (about ten in each
    of two layers, in either direction), each time by 2^-9 / sqrt(3) of itself
    or less in the mean: sqrt(40) 2^-9 / sqrt(3) = 0.7% where the errors are
    independent, 8% where all add up.  A tensor's gradient has to be within 8%
    in the norm."""
    heads, vocab, lengths, tau = 2, 301, (37, 1, 64, 150), 2.0
    p = ex.make_parameters(2, 64, vocab, max(lengths))
    b = ex.make_batch(lengths, vocab, 16, 7)
    for t in p.values():
        t.requires_grad_()
    z = ex.logits_of(p, b["tokens"], b["positions"], b["cu_seqlens"], heads)
    loss = ex.distill_loss(z, b["teacher_index"], b["teacher_logits"], tau).mean()
    got = dict(zip(p, torch.autograd.grad(loss, list(p.values()))))
    p64 = {n: t.detach().double().cpu().requires_grad_() for n, t in p.items()}
    b64 = {n: t.cpu() for n, t in b.items()}
    z64 = ex.logits_of(p64, b64["tokens"], b64["positions"], b64["cu_seqlens"], heads, torch.float64, plain_norm,
                       plain_attention)
    loss64 = plain_loss(z64, b64, tau)
    want = dict(zip(p64, torch.autograd.grad(loss64, list(p64.values()))))
    assert abs(loss.item() - loss64.item()) <= 0.01 * loss64.item()
    for n in p:
        w = want[n].numpy()
        off = np.linalg.norm(got[n].double().cpu().numpy() - w)
        if n.endswith("c_attn.bias"):
            # the part for the keys shifts all scores of a row alike: its gradient is zero, and what is found is rounding
            width = w.size // 3
            assert np.abs(w[width:2 * width]).max() <= 1e-12
        assert off <= 0.08 * np.linalg.norm(w), (n, off, np.linalg.norm(w))


def test_ranks_stay_equal_and_losses_fall(ex):
    models, losses = ex.run(ranks=3, steps=4, layers=1, heads=2, width=128, vocab=1009, top=8, lengths=(40, 90))
    for m in models[1:]:
        for a, b in zip(models[0].values(), m.values()):
            assert torch.equal(a, b)
    assert all(np.isfinite(losses).ravel())
    assert all(after < before for before, after in zip(losses[0], losses[-1]))


def test_one_rank_alone_and_again_gives_the_same_bits(ex):
    size = dict(steps=2, layers=1, heads=2, width=128, vocab=1009, top=8, lengths=(40, 90))
    first, losses = ex.run(ranks=1, **size)
    again, losses2 = ex.run(ranks=1, **size)
    assert losses == losses2
    for a, b in zip(first[0].values(), again[0].values()):
        assert torch.equal(a, b)
