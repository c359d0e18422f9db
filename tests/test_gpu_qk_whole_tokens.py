"""ar_qk_norm_rope and its gradient with rotation where there are enough tokens
that warps take whole ones, against the formulas in 64 bits on the device.

Tolerances: u of the result's type for its rounding, 2^-18 of the magnitudes for
binary32's arithmetic forward and twice that backward (a head's sums of at most
256 products, 24 units of 2^-24; a reciprocal square root, products, sines and
cosines off by 2 units and angles by 2^-30: below 64 units).  A weight's
gradient sums heads x tokens rows, each warp those of its tokens one after
another: at most 12001 * 10 / 1200 = 100 here, some 20 levels after that and the
term's own 64 units: 256 units, 2^-16, of the terms' magnitudes.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
TOKENS = 12001  # more than four to a warp of 304 blocks of eight


@pytest.fixture(scope="module")
def ar():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import binding
    torch.cuda.set_device(0)
    return binding


def within(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), bad.nonzero()[:3].tolist())


def turned(x, angle, rotary, interleaved, sign=1):
    y, size = x.clone(), x.abs()
    a, b = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, rotary // 2), slice(rotary // 2, rotary))
    c, s = torch.cos(angle)[:, None], sign * torch.sin(angle)[:, None]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


# vectors of 16 and of 8 bytes, one element at a time (18; 62 in half), all of a head or a part of it
CASES = [("bf16", 128, 128, 4, 2), ("f32", 64, 32, 3, 3), ("f16", 64, 64, 10, 1), ("f32", 18, 18, 2, 1),
         ("bf16", 62, 20, 3, 2), ("f16", 24, 8, 5, 0), ("f32", 128, 64, 1, 4), ("bf16", 256, 256, 2, 1)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,dim,rotary,heads,kv", CASES)
def test_rotation(ar, dtype, dim, rotary, heads, kv, interleaved):
    g = torch.Generator(device="cuda")
    g.manual_seed(dim + heads)

    def tensors():
        return [torch.randn(TOKENS, n, dim, device="cuda", generator=g).to(DT[dtype]) if n else None for n in (heads, kv)]

    xs, ups = tensors(), tensors()
    ws = [1 + 0.3 * torch.randn(dim, device="cuda", generator=g) if n else None for n in (heads, kv)]
    # every token a position of its own, out of order, far ones and negative ones among them
    pos = torch.randint(-100000, 1000000, (TOKENS,), device="cuda", generator=g, dtype=torch.int32)
    freq = torch.tensor([10000.0 ** (-2 * i / rotary) for i in range(rotary // 2)], dtype=torch.float64, device="cuda")
    angle = pos.double()[:, None] * freq  # off by 2^-53 of 1e6: 2^-33
    how = dict(rotary_dim=rotary, interleaved=interleaved, eps=1e-6)
    outs, grads = ([None if x is None else torch.full_like(x, 7.0) for x in xs] for _ in range(2))
    ar.check(ar.ar_qk_norm_rope(*xs, *ws, pos, *outs, **how), "forward")
    dws = [None if w is None else torch.full_like(w, 7.0) for w in ws]
    workspace = torch.empty(ar.ar_qk_norm_rope_workspace_bytes(TOKENS, heads, kv, dim), dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_qk_norm_rope_backward(*ups, *xs, *ws, pos, *grads, *dws, workspace, **how), "backward")
    for x, up, w, out, dx, dw in zip(xs, ups, ws, outs, grads, dws):
        if x is None:
            continue
        x, w = x.double(), w.double()
        rstd = (x.square().mean(2, keepdim=True) + 1e-6).rsqrt()
        want, size = turned(x * rstd * w, angle, rotary, interleaved)
        within(out, want, U[dtype] * want.abs() + 2.0 ** -18 * size + TINY[dtype], "out")
        turn_back, size = turned(up.double(), angle, rotary, interleaved, -1)
        xh = x * rstd
        want = rstd * (turn_back * w - xh * (turn_back * w * xh).mean(2, keepdim=True))
        sizes = rstd * (size * w.abs() + xh.abs() * (size * (w * xh).abs()).mean(2, keepdim=True))
        within(dx, want, U[dtype] * want.abs() + 2.0 ** -17 * sizes + TINY[dtype], "dx")
        within(dw, (turn_back * xh).sum((0, 1)), 2.0 ** -16 * (size * xh.abs()).sum((0, 1)), "dw")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f32", 64), ("f32", 18)])
def test_gradients_of_many_tokens_are_as_those_of_few(ar, dtype, dim, interleaved):
    """Each token's gradient has the bits of a call on its neighbours and it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(dim)
    xs, ups = ([torch.randn(TOKENS, n, dim, device="cuda", generator=g).to(DT[dtype]) for n in (5, 2)] for _ in range(2))
    ws = [1 + 0.3 * torch.randn(dim, device="cuda", generator=g) for _ in range(2)]
    pos = torch.randint(-100000, 1000000, (TOKENS,), device="cuda", generator=g, dtype=torch.int32)

    def gradients(a, b):
        to = [torch.empty(b - a, n, dim, dtype=DT[dtype], device="cuda") for n in (5, 2)]
        ar.check(ar.ar_qk_norm_rope_backward(*(u[a:b] for u in ups), *(x[a:b] for x in xs), *ws, pos[a:b], *to, None, None,
                                             interleaved=interleaved), "backward")
        return to

    all_ = gradients(0, TOKENS)
    for a in (0, 1, 2432, 4863, 7777, TOKENS - 10):
        assert all(torch.equal(x[a:a + 10], y) for x, y in zip(all_, gradients(a, a + 10)))
