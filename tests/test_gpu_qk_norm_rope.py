"""ar_qk_norm_rope and its gradient against the formulas in 64 bits.

Tolerances.  u is the unit roundoff of the result's type (2^-24 f32, 2^-8 bf16,
2^-11 f16): one rounding of a result costs at most u of it.  What comes before is
binary32: a head's sum of at most 256 squares or products (8 in a lane's chain
and as many levels, or 16 and 5: at most 24 units of 2^-24), a reciprocal square
root (2 units), a few products, and sines and cosines that are off by 2^-23 of
one: together below 64 units, 2^-18, of the magnitudes involved.  A weight's
gradient sums at most 600 rows here, at most 75 of them in one chain (a warp's
run), and some 10 levels after it: 128 units with the term's own error.
The angle is exact to 2^-34 turns in the kernel; its frequency is a binary64
number, off by 2^-51 at most (a power, a quotient and their libraries), which at
position 2^31 is 2^-20.
"""
from fractions import Fraction
import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
ARITH = 2.0 ** -18
SUMS = 2.0 ** -16
# 2 pi to 50 digits
TURN = Fraction(628318530717958647692528676655900576839433879875021, 10 ** 50)


@pytest.fixture(scope="module")
def ar():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import binding
    torch.cuda.set_device(0)
    return binding


def f64(t):
    return t.double().cpu().numpy()


def within(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3])


def make(tokens, heads, kv, dim, dtype, seed, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(tokens, h, dim, device="cuda", generator=g) * spread).to(DT[dtype]) for h in (heads, kv)]


def weights(dim, params, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(1 + 0.3 * torch.randn(dim, device="cuda", generator=g)).to(DT[params]) for _ in range(2)]


def angles(positions, rotary, base, frequencies):
    """[tokens, rotary / 2], reduced to one turn without any rounding before."""
    f = frequencies if frequencies is not None else [float(base) ** (-2 * i / rotary) for i in range(rotary // 2)]
    turns = [[float(Fraction(x) * int(p) / TURN % 1) for x in f] for p in positions]
    return 2 * np.pi * np.array(turns).reshape(len(positions), rotary // 2)


def turned(x, angle, rotary, interleaved, sign=1):
    """x with its pairs turned, and the sum of the magnitudes that each result is made of."""
    y, size = x.copy(), np.abs(x)
    a, b = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, rotary // 2), slice(rotary // 2, rotary))
    c, s = np.cos(angle)[:, None], sign * np.sin(angle)[:, None]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    both = np.abs(x[..., a]) + np.abs(x[..., b])
    size[..., a] = size[..., b] = both
    return y, size


def check(ar, xs, ws, positions, dtype, params, ups=None, outs=None, rotary=None, base=10000.0, frequencies=None,
          interleaved=False, eps=1e-6, grads=None):
    dim = xs[0].shape[2]
    r = dim if rotary is None else rotary
    how = dict(rotary_dim=rotary, base=base, frequencies=frequencies, interleaved=interleaved, eps=eps)
    angle = angles(positions.tolist(), r, base, frequencies)
    given = [f64(x) if x is not None else None for x in xs]
    if outs is None:
        outs = [None if x is None else torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda") for x in xs]
    if ups is None:
        ar.check(ar.ar_qk_norm_rope(xs[0], xs[1], ws[0], ws[1], positions, outs[0], outs[1], **how), "ar_qk_norm_rope")
        for x, w, out in zip(given, ws, outs):
            if x is None:
                continue
            n = x / np.sqrt((x * x).mean(2, keepdims=True) + np.float32(eps)) * (1.0 if w is None else f64(w))
            want, size = turned(n, angle, r, interleaved)
            within(f64(out), want, U[dtype] * np.abs(want) + ARITH * size + TINY[dtype], "out")
        return outs
    up64 = [None if x is None else f64(x) for x in ups]
    dws = [torch.full((dim,), 7.0, dtype=DT[params], device="cuda") for _ in xs]
    if grads is None:
        grads = [None if x is None else torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda") for x in xs]
    ws_bytes = ar.ar_qk_norm_rope_workspace_bytes(xs[0].shape[0], xs[0].shape[1], 0 if xs[1] is None else xs[1].shape[1], dim)
    workspace = torch.full((ws_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_qk_norm_rope_backward(ups[0], ups[1], xs[0], xs[1], ws[0], ws[1], positions, grads[0], grads[1],
                                         dws[0], dws[1], workspace, **how), "ar_qk_norm_rope_backward")
    for x, up, w, dx, dw in zip(given, up64, ws, grads, dws):
        if x is None:
            assert (dw == 0).all()
            continue
        w64 = np.ones(dim) if w is None else f64(w)
        rstd = 1 / np.sqrt((x * x).mean(2, keepdims=True) + np.float32(eps))
        xh = x * rstd
        g, size = turned(up, angle, r, interleaved, -1)
        want = rstd * (g * w64 - xh * (g * w64 * xh).mean(2, keepdims=True))
        sizes = rstd * (size * np.abs(w64) + np.abs(xh) * (size * np.abs(w64 * xh)).mean(2, keepdims=True))
        within(f64(dx), want, U[dtype] * np.abs(want) + 2 * ARITH * sizes + TINY[dtype], "dx")
        want = (g * xh).sum((0, 1))
        within(f64(dw), want, U[params] * np.abs(want) + SUMS * (size * np.abs(xh)).sum((0, 1)) + TINY[params], "dw")
    return grads, dws


def positions_of(tokens, first=0):
    return (torch.arange(tokens, device="cuda") + first).to(torch.int32)


@pytest.mark.parametrize("dtype,params", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (64, 32), (128, 128), (80, 40), (32, 32), (256, 64)])
def test_types_and_sizes(ar, dtype, params, interleaved, dim, rotary):
    for tokens, heads, kv in ((3, 4, 2), (37, 5, 1)):
        xs, ws = make(tokens, heads, kv, dim, dtype, 1), weights(dim, params, 2)
        ups = make(tokens, heads, kv, dim, dtype, 3)
        check(ar, xs, ws, positions_of(tokens, 5), dtype, params, rotary=rotary, interleaved=interleaved)
        check(ar, xs, ws, positions_of(tokens, 5), dtype, params, ups, rotary=rotary, interleaved=interleaved)


@pytest.mark.parametrize("dim,rotary", [(2, 2), (2, 0), (6, 4), (10, 10), (18, 6), (62, 62), (72, 8), (130, 2), (254, 254),
                                        (256, 256), (256, 0), (96, 48), (120, 120)])
def test_odd_head_sizes(ar, dim, rotary):
    for dtype, interleaved in itertools.product(("bf16", "f32"), (False, True)):
        xs, ws = make(20, 3, 2, dim, dtype, 4), weights(dim, "f32", 5)
        check(ar, xs, ws, positions_of(20), dtype, "f32", rotary=rotary, interleaved=interleaved)
        check(ar, xs, ws, positions_of(20), dtype, "f32", make(20, 3, 2, dim, dtype, 6), rotary=rotary, interleaved=interleaved)


@pytest.mark.parametrize("tokens,heads,kv", [(1, 1, 1), (1, 32, 8), (2, 12, 12), (600, 1, 1), (200, 3, 0), (23, 25, 25), (5, 100, 3)])
def test_heads_and_tokens(ar, tokens, heads, kv):
    """Also keys that there are none of, and fewer rounds than warps."""
    xs, ws = make(tokens, heads, max(kv, 1), 64, "bf16", 7), weights(64, "f32", 8)
    ups = make(tokens, heads, max(kv, 1), 64, "bf16", 9)
    if not kv:
        xs[1] = ups[1] = ws[1] = None
    check(ar, xs, ws, positions_of(tokens), "bf16", "f32")
    check(ar, xs, ws, positions_of(tokens), "bf16", "f32", ups)


def test_many_tokens_are_as_few(ar):
    """More rounds than all warps together: each token's result has the bits of
    a call on it alone."""
    xs, ws = make(9000, 9, 2, 128, "bf16", 10), weights(128, "f32", 11)
    pos = positions_of(9000, 300000)
    outs = [torch.empty_like(x) for x in xs]
    ar.check(ar.ar_qk_norm_rope(*xs, *ws, pos, *outs), "all")
    for a in (0, 1, 4321, 8990):
        few = [torch.empty_like(x[a:a + 10]) for x in xs]
        ar.check(ar.ar_qk_norm_rope(*(x[a:a + 10] for x in xs), *ws, pos[a:a + 10], *few), "few")
        assert all(torch.equal(x[a:a + 10], y) for x, y in zip(outs, few))


@pytest.mark.parametrize("heads,kv", [(4, 0), (60, 1), (1, 60), (3, 3)])
def test_whole_tokens_to_a_warp(ar, heads, kv):
    """Enough tokens that warps take whole ones; keys that there are none of, or
    few, and as many blocks as the workspace has rows.  (A weight's gradient is
    summed over up to 60 x 10001 rows, in chains of at most 10001 * 60 / 2400 =
    250: 512 units of 2^-24 with its terms'.)"""
    global SUMS
    xs, ups, ws = make(10001, heads, max(kv, 1), 16, "f16", 42), make(10001, heads, max(kv, 1), 16, "f16", 43), weights(16, "f32", 44)
    if not kv:
        xs[1] = ups[1] = ws[1] = None
    pos = positions_of(10001)
    check(ar, xs, ws, pos, "f16", "f32", rotary=0)
    before, SUMS = SUMS, 2.0 ** -15
    try:
        check(ar, xs, ws, pos, "f16", "f32", ups, rotary=0)
    finally:
        SUMS = before


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(ar, interleaved):
    """Angles are as exact at 2^31 as at 0, below it and before it too."""
    pos = torch.tensor([0, 1, -1, 4095, 131071, 10 ** 6, 16777217, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    xs, ws = make(9, 2, 1, 64, "f32", 12), weights(64, "f32", 13)
    check(ar, xs, ws, pos, "f32", "f32", interleaved=interleaved)
    check(ar, xs, ws, pos, "f32", "f32", make(9, 2, 1, 64, "f32", 14), interleaved=interleaved)


def test_frequencies(ar):
    g = np.random.Generator(np.random.PCG64(15))
    xs, ws = make(33, 2, 2, 48, "f32", 16), weights(48, "f32", 17)
    freq = [0.0, -1.0, -1e-30, 7.25] + list(g.uniform(0, 10, 12))
    check(ar, xs, ws, positions_of(33, 70000), "f32", "f32", rotary=32, frequencies=freq, base=-1.0)
    # those of the base, given one by one, are the base's
    own = [500.0 ** (-2 * i / 48) for i in range(24)]
    a = check(ar, xs, ws, positions_of(33), "f32", "f32", base=500.0)
    b = check(ar, xs, ws, positions_of(33), "f32", "f32", frequencies=own)
    assert all((x - y).abs().max() <= 2e-6 for x, y in zip(a, b))


def test_bases_by_turns(ar):
    """A call takes its own base, whatever the one before had."""
    xs, ws = make(20, 2, 1, 64, "f32", 18), weights(64, "f32", 19)
    for base, rotary in ((10000.0, 64), (500000.0, 64), (10000.0, 32), (500000.0, 32), (10000.0, 64)):
        check(ar, xs, ws, positions_of(20, 1000), "f32", "f32", base=base, rotary=rotary)


@pytest.mark.parametrize("layout", ["one projection", "heads outside", "padded", "odd start", "odd stride"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layouts(ar, layout, dtype):
    t, h, kv, d = 45, 4, 2, 64

    def place(parts):
        if layout == "one projection":
            return list(torch.split(torch.cat(parts, 1).contiguous(), [p.shape[1] for p in parts], 1))
        if layout == "heads outside":
            return [p.transpose(0, 1).contiguous().transpose(0, 1) for p in parts]
        if layout == "padded":
            return [torch.nn.functional.pad(p, (0, 8, 0, 1))[:, :-1, :d] for p in parts]
        if layout == "odd start":
            return [torch.nn.functional.pad(p, (1, 7))[..., 1:1 + d] for p in parts]
        return [torch.nn.functional.pad(p, (0, 3))[..., :d] for p in parts]

    xs, ups, ws = place(make(t, h, kv, d, dtype, 20)), place(make(t, h, kv, d, dtype, 21)), weights(d, "f32", 22)
    seven = [torch.full((t, n, d), 7.0, dtype=DT[dtype], device="cuda") for n in (h, kv)]
    check(ar, xs, ws, positions_of(t), dtype, "f32", outs=place(seven))
    check(ar, xs, ws, positions_of(t), dtype, "f32", ups, grads=place(seven))


def test_in_place(ar):
    xs, ws, ups = make(50, 4, 2, 64, "bf16", 23), weights(64, "f32", 24), make(50, 4, 2, 64, "bf16", 25)
    outs = check(ar, xs, ws, positions_of(50), "bf16", "f32")
    grads, dws = check(ar, xs, ws, positions_of(50), "bf16", "f32", ups)
    both = torch.cat(xs, 1)
    parts = both.split((4, 2), 1)
    ar.check(ar.ar_qk_norm_rope(*parts, *ws, positions_of(50), *parts), "in place")
    assert all(torch.equal(a, b) for a, b in zip(parts, outs))
    ws_ = torch.empty(ar.ar_qk_norm_rope_workspace_bytes(50, 4, 2, 64), dtype=torch.uint8, device="cuda")
    for over_up in (True, False):
        x, up = torch.cat(xs, 1).split((4, 2), 1), [u.clone() for u in ups]
        to = up if over_up else x
        dw = [torch.empty(64, device="cuda") for _ in ws]
        ar.check(ar.ar_qk_norm_rope_backward(*up, *x, *ws, positions_of(50), *to, *dw, ws_), "in place")
        assert all(torch.equal(a, b) for a, b in zip((*to, *dw), (*grads, *dws)))


def test_without_weights(ar):
    xs, ups = make(31, 3, 1, 64, "f16", 26), make(31, 3, 1, 64, "f16", 27)
    check(ar, xs, [None, None], positions_of(31), "f16", "f16")
    check(ar, xs, [None, None], positions_of(31), "f16", "f16", ups)
    grads = [torch.empty_like(x) for x in xs]
    want, _ = check(ar, xs, [None, None], positions_of(31), "f16", "f16", ups)
    ar.check(ar.ar_qk_norm_rope_backward(*ups, *xs, None, None, positions_of(31), *grads, None, None), "no weights")
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


def test_rows_of_zeros_and_large_rows(ar):
    """A row of zeros is zeros (eps keeps it from a division by zero), its
    gradient the upstream one times eps^-1/2; squares near binary32's end."""
    xs, ws, ups = make(12, 2, 1, 64, "f32", 28), weights(64, "f32", 29), make(12, 2, 1, 64, "f32", 30)
    xs[0][3] = 0
    xs[0][5] *= 1e17
    xs[1][7] *= 1e-17
    out = check(ar, xs, ws, positions_of(12), "f32", "f32", eps=1e-5)
    assert (out[0][3] == 0).all()
    check(ar, xs, ws, positions_of(12), "f32", "f32", ups, eps=1e-5)


def test_one_bad_row_stays_one(ar):
    xs, ws = make(40, 4, 2, 128, "bf16", 31), weights(128, "f32", 32)
    outs = check(ar, xs, ws, positions_of(40), "bf16", "f32")
    for bad in (float("nan"), float("inf")):
        x = [t.clone() for t in xs]
        x[0][17, 2, 5] = bad
        got = [torch.empty_like(t) for t in x]
        ar.check(ar.ar_qk_norm_rope(*x, *ws, positions_of(40), *got), "bad row")
        same = got[0] == outs[0]
        assert not same[17, 2].any()
        same[17, 2] = True
        assert same.all() and torch.equal(got[1], outs[1])


def test_gradient_agrees_with_differences(ar):
    """Against central differences of the formula in 64 bits: at a step of 1e-4
    their own error is below 1e-6 of the terms; f32 gradients' is below 2^-17."""
    xs, ws, ups, pos = make(7, 3, 2, 16, "f32", 33), weights(16, "f32", 34), make(7, 3, 2, 16, "f32", 35), positions_of(7, 3)
    grads, dws = check(ar, xs, ws, pos, "f32", "f32", ups, rotary=12)
    angle = angles(pos.tolist(), 12, 10000.0, None)

    def total(x, w):
        return sum((turned(a / np.sqrt((a * a).mean(2, keepdims=True) + np.float32(1e-6)) * b, angle, 12, False)[0] * f64(u)).sum()
                   for a, b, u in zip(x, w, ups))

    g = np.random.Generator(np.random.PCG64(36))
    x, w, h = [f64(t) for t in xs], [f64(t) for t in ws], 1e-4
    for _ in range(5):
        dx, dw = [g.standard_normal(t.shape) for t in x], [g.standard_normal(t.shape) for t in w]
        move = lambda s: total([a + s * h * b for a, b in zip(x, dx)], [a + s * h * b for a, b in zip(w, dw)])  # noqa: E731
        terms = [(f64(a) * b) for a, b in zip((*grads, *dws), (*dx, *dw))]
        assert abs((move(1) - move(-1)) / (2 * h) - sum(t.sum() for t in terms)) <= 2.0 ** -16 * sum(np.abs(t).sum() for t in terms)


def test_same_bits_on_another_stream_and_in_graphs(ar):
    """Also two graphs that share a workspace, replayed one after the other."""
    xs, ws, ups, pos = make(500, 6, 2, 64, "bf16", 37), weights(64, "f32", 38), make(500, 6, 2, 64, "bf16", 39), positions_of(500)
    outs = check(ar, xs, ws, pos, "bf16", "f32")
    grads, dws = check(ar, xs, ws, pos, "bf16", "f32", ups)
    ups2 = [u * 2 for u in ups]
    grads2, dws2 = check(ar, xs, ws, pos, "bf16", "f32", ups2)
    workspace = torch.empty(ar.ar_qk_norm_rope_workspace_bytes(500, 6, 2, 64), dtype=torch.uint8, device="cuda")
    got, graphs = [], []
    for up in (ups, ups2):
        to = [torch.zeros_like(x) for x in (*outs, *grads, *dws)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ar.check(ar.ar_qk_norm_rope(*xs, *ws, pos, *to[:2]), "forward")
            ar.check(ar.ar_qk_norm_rope_backward(*up, *xs, *ws, pos, *to[2:], workspace), "backward")
        got.append(to)
        graphs.append(graph)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for x in got[0] + got[1]:
            x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for graph in graphs:
                graph.replay()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[0], (*outs, *grads, *dws)))
        assert all(torch.equal(a, b) for a, b in zip(got[1], (*outs, *grads2, *dws2)))


def test_refusals(ar):
    xs, ws, pos = make(20, 4, 2, 64, "bf16", 40), weights(64, "f32", 41), positions_of(20)
    q, k = xs
    o, p = torch.empty_like(q), torch.empty_like(k)
    bad, unsupported, call = ar.AR_ERR_INVALID_ARG, ar.AR_ERR_UNSUPPORTED, ar.ar_qk_norm_rope
    launches = ar.ar_kernel_launches()
    assert call(q.int(), k.int(), *ws, pos, o.int(), p.int()) == unsupported
    assert call(q, k, ws[0].half(), ws[1].half(), pos, o, p) == unsupported       # bf16 heads, f16 weights
    assert call(q, k, ws[0], ws[1].bfloat16(), pos, o, p) == bad                  # two types of weights
    assert call(q, k.half(), *ws, pos, o, p.half()) == bad
    assert call(q, k[:19], *ws, pos, o, p[:19]) == bad and call(q, k, *ws, pos[:19], o, p) == bad
    assert call(q, k, *ws, pos.long(), o, p) == bad and call(q, k, *ws, pos.cpu(), o, p) == bad
    assert call(q, k, ws[0][:32], ws[1], pos, o, p) == bad and call(q, k, *ws, pos, o[..., :32], p) == bad
    assert call(q, None, *ws, pos, o, p) == bad and call(q, k, *ws, pos, o, None) == bad
    assert call(q, k, *ws, pos, o, p, rotary_dim=65) == bad and call(q, k, *ws, pos, o, p, rotary_dim=66) == bad
    assert call(q, k, *ws, pos, o, p, frequencies=[1.0] * 31) == bad
    assert call(q, k, *ws, pos, o, p, frequencies=[float("nan")] * 32) == bad
    assert call(q, k, *ws, pos, o, p, base=0.0) == bad and call(q, k, *ws, pos, o, p, eps=-1.0) == bad
    assert call(q[..., ::2], k[..., ::2], ws[0][:32], ws[1][:32], pos, o[..., :32], p[..., :32]) == bad
    assert call(q, k, *ws, pos, k.repeat(1, 2, 1)[:, :4].expand(20, 4, 64)[:1].expand(20, 4, 64), p) == bad
    assert call(q, k, *ws, pos, o, o[:, :2]) == bad                                # both into one place
    assert ar.ar_kernel_launches() == launches
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((64,), 7.0, device="cuda")
    assert call(none, none[:, :2], *ws, pos[:0], none, none[:, :2]) == ar.AR_OK
    assert ar.ar_qk_norm_rope_backward(none, none[:, :2], none, none[:, :2], *ws, pos[:0], none, none[:, :2], dw, None) == ar.AR_OK
    assert ar.ar_kernel_launches() == launches and (dw == 0).all()
