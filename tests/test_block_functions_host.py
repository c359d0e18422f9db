"""qk_norm_rope, diff_attention and activation8_linear as PyTorch functions, with
the library's calls replaced by their formulas: no device is needed."""
import types

import pytest

torch = pytest.importorskip("torch")

EPS = 1e-6


@pytest.fixture
def ex(monkeypatch):
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import distill_step

    def turned(x, positions, sign=1):
        n = x.shape[2] // 2
        angle = positions.float()[:, None, None] * 100.0 ** (-torch.arange(n) / n)
        c, s, a, b = torch.cos(angle), sign * torch.sin(angle), x[..., :n], x[..., n:]
        return torch.cat((a * c - b * s, b * c + a * s), 2)

    def rope(q, k, q_weight, k_weight, positions, q_out, k_out, **how):
        for x, w, y in ((q, q_weight, q_out), (k, k_weight, k_out)):
            y.copy_(turned(x * (x.square().mean(2, keepdim=True) + EPS).rsqrt() * w, positions))

    def rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, dq, dk, dq_weight, dk_weight, workspace, **how):
        for dy, x, w, dx, dw in ((dq_out, q, q_weight, dq, dq_weight), (dk_out, k, k_weight, dk, dk_weight)):
            r = (x.square().mean(2, keepdim=True) + EPS).rsqrt()
            g = turned(dy, positions, -1)
            dw.copy_((g * x * r).sum((0, 1)))
            dx.copy_(r * (g * w - x * r * r * (g * w * x).mean(2, keepdim=True)))

    def scores(q, k):  # one sequence, as many heads of k as of q
        s = torch.einsum("ihd,jhd->hij", q, k) * q.shape[2] ** -0.5
        return s.masked_fill(torch.ones(len(q), len(q), dtype=torch.bool).triu(1), -float("inf"))

    def attention(q, k, v, lam, cu_seqlens, out, second, lse):
        s = scores(q, k)
        lse.copy_(s.logsumexp(2))
        p = s.softmax(2)
        second.copy_(torch.einsum("hij,jhd->ihd", p[1::2], v))
        out.copy_(torch.einsum("hij,jhd->ihd", p[::2], v) - lam[:, None] * second)

    def attention_backward(dout, q, k, v, lam, out, second, lse, cu_seqlens, dq, dk, dv, dlam, workspace):
        p = (scores(q, k) - lse[:, :, None]).exp()
        dp = torch.einsum("ihd,jhd->hij", dout, v)
        d1 = (dout * second).sum(2).t()
        d0 = (dout * out).sum(2).t() + lam[:, None] * d1
        ds = torch.empty_like(p)
        ds[::2] = p[::2] * (dp - d0[:, :, None])
        ds[1::2] = -lam[:, None, None] * p[1::2] * (dp - d1[:, :, None])
        ds *= q.shape[2] ** -0.5
        dq.copy_(torch.einsum("hij,jhd->ihd", ds, k))
        dk.copy_(torch.einsum("hij,ihd->jhd", ds, q))
        dv.copy_(torch.einsum("hij,ihd->jhd", p[::2] - lam[:, None, None] * p[1::2], dout))
        dlam.copy_(-d1.sum(1))

    def act(x):
        return x * torch.sigmoid(1.702 * x)

    kept = []  # what was packed, its number in the scales

    def pack(x, y, codes, scales, kind):
        y.copy_(act(x))
        scales[0, 0] = len(kept)
        kept.append(x.detach().clone())

    def unpack(codes, scales, dy, dx, y, kind):
        x = kept[int(scales[0, 0])]
        s = torch.sigmoid(1.702 * x)
        y.copy_(act(x))
        dx.copy_(dy * (s + 1.702 * x * s * (1 - s)))

    fake = types.SimpleNamespace(
        check=lambda *a: None, ACTIVATION8_BLOCK=128, ar_qk_norm_rope=rope, ar_qk_norm_rope_backward=rope_backward,
        ar_qk_norm_rope_workspace_bytes=lambda *a: 16, ar_diff_attention=attention,
        ar_diff_attention_backward=attention_backward, ar_diff_attention_workspace_bytes=lambda *a: 16)

    fake.ar_activation8, fake.ar_activation8_backward = pack, unpack
    monkeypatch.setattr(distill_step, "ar", fake)
    return distill_step


def cases(ex):
    g = torch.Generator()
    g.manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g).requires_grad_()

    positions, cu = torch.arange(5, dtype=torch.int32), torch.tensor([0, 6], dtype=torch.int32)
    return {"qk_norm_rope": (lambda q, k, a, b: torch.cat(ex.qk_norm_rope(q, k, a, b, positions, interleaved=False), 1),
                             (normal(5, 3, 8), normal(5, 2, 8), normal(8), normal(8))),
            "diff_attention": (lambda q, k, v, lam: ex.diff_attention(q, k, v, lam, cu),
                               (normal(6, 4, 8), normal(6, 4, 8), normal(6, 2, 8), normal(2))),
            "activation8_linear": (ex.activation8_linear, (normal(5, 9), normal(9, 4), normal(4)))}


NAMES = ["qk_norm_rope", "diff_attention", "activation8_linear"]


@pytest.mark.parametrize("name", NAMES)
def test_first_derivatives(ex, name):
    """Against differences of the replaced calls in 32 bits: off by 1e-3 of the
    magnitudes at a step of 1e-2 (its cube's third and binary32's rounding)."""
    f, inputs = cases(ex)[name]
    y = f(*inputs)
    g = torch.Generator()
    g.manual_seed(2)
    up = torch.randn(y.shape, generator=g)
    grads = torch.autograd.grad(y, inputs, up)
    h = 1e-2
    d = [torch.randn(x.shape, generator=g) for x in inputs]
    with torch.no_grad():
        plus, minus = (f(*(x + s * h * e for x, e in zip(inputs, d))) for s in (1, -1))
    want = ((plus.double() - minus.double()) * up / (2 * h)).sum()
    got = sum((a * e).sum() for a, e in zip(grads, d))
    size = sum((a * e).abs().sum() for a, e in zip(grads, d))
    assert abs(want - got) <= 1e-3 * size


@pytest.mark.parametrize("name", NAMES)
def test_second_derivatives_are_refused(ex, name):
    f, inputs = cases(ex)[name]
    loss = f(*inputs).square().sum()
    grads = torch.autograd.grad(loss, inputs, create_graph=True)
    penalty = sum(g.square().sum() for g in grads) + sum(x.square().sum() for x in inputs)
    for x in inputs:
        with pytest.raises(RuntimeError, match="second derivatives"):
            torch.autograd.grad(penalty, x, retain_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        penalty.backward()


@pytest.mark.parametrize("name", NAMES)
def test_a_graph_of_the_gradients_alone_changes_nothing(ex, name):
    f, inputs = cases(ex)[name]
    y = f(*inputs)
    plain = torch.autograd.grad(y.sum(), inputs, retain_graph=True)
    graphed = torch.autograd.grad(y.sum(), inputs, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, graphed))


def test_an_output_that_is_not_used_has_a_zero_gradient(ex):
    f, (q, k, a, b) = cases(ex)["qk_norm_rope"]
    q_out, _ = ex.qk_norm_rope(q, k, a, b, torch.arange(5, dtype=torch.int32))
    dk, db = torch.autograd.grad(q_out.square().sum(), (k, b))
    assert (dk == 0).all() and (db == 0).all()


def test_parameters_of_both_blocks(ex):
    """Those of GPT-2 are as they were without the choice; the other block's have
    the norms', no table of positions."""
    plain = ex.make_parameters(2, 32, 50, 9, device="cpu")
    same = ex.make_parameters(2, 32, 50, 9, device="cpu", block="gpt2", heads=4)
    assert plain.keys() == same.keys() and all(torch.equal(plain[n], same[n]) for n in plain)
    other = ex.make_parameters(2, 32, 50, 9, device="cpu", block="diff", heads=2)
    assert other.keys() - plain.keys() == {f"h.{i}.{n}" for i in (0, 1) for n in ("q_norm.weight", "k_norm.weight", "lambda")}
    assert plain.keys() - other.keys() == {"wpe"}
    assert other["h.1.q_norm.weight"].shape == (8,) and other["h.0.lambda"].shape == (2,)
