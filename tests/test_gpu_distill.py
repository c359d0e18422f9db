"""ar_distill_loss and ar_distill_loss_backward against the formula in 64 bits.

Tolerances.  u is the unit roundoff of the result's type, and the arithmetic
before the one rounding to it is binary32 (unit 2^-24).  An exponent z/tau -
lse is off by a few units of |z|/tau + |lse| (below 64 in these tests, but for
the rows that are made extreme), so a probability by at most 2^-16 of itself; a
loss adds terms p (log p - z/tau + lse) whose magnitudes are known: 2^-18 of
their sum; lse: 2^-18 of its terms.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}


@pytest.fixture(scope="module")
def ar():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from allreduce_gradient_reduction_gb300 import build as b
    b.build()
    from allreduce_gradient_reduction_gb300 import binding
    torch.cuda.set_device(0)
    return binding


def rows_of(values, dtype, pad=0, offset=0):
    r, c = values.shape
    flat = torch.full((offset + r * (c + pad),), float("nan"), dtype=DT[dtype], device="cuda")
    m = flat[offset:].view(r, c + pad)[:, :c]
    m.copy_(torch.from_numpy(values))
    return m


def make(rows, vocab, top, dtype, seed, pad=0, offset=0, vdtype="f32"):
    g = np.random.Generator(np.random.PCG64(seed))
    z = rows_of(g.standard_normal((rows, vocab)) * 2, dtype, pad, offset)
    index = torch.from_numpy(g.integers(0, vocab, (rows, top)).astype(np.int32)).cuda()  # words may repeat
    value = torch.from_numpy(g.standard_normal((rows, top)) * 2).to("cuda", DT[vdtype])
    scale = torch.from_numpy(g.uniform(0.5, 1.5, rows)).float().cuda()
    return z, index, value, scale


def f64(t):
    return t.double().cpu().numpy()


def formula(z, index, value, scale, tau, lse=None):
    """(loss, lse, dlogits, magnitude of the loss's terms, of the gradient's, whether the row is live) in 64 bits."""
    Z, I, V = f64(z) / tau, index.cpu().numpy(), f64(value) / tau
    rows, vocab = Z.shape
    with np.errstate(invalid="ignore", divide="ignore"):
        V = np.where((I >= 0) & (I < vocab), V, -np.inf)
        if V.shape[1]:
            top = V.max(1, keepdims=True)
            E = np.exp(V - np.where(np.isfinite(top), top, 0))
        else:
            E = np.zeros((rows, 0))
        total = E.sum(1, keepdims=True)
        live = total[:, 0] > 0
        P = np.where(live[:, None], E / np.where(total > 0, total, 1), 0)
        zmax = Z.max(1, keepdims=True)
        own = (zmax + np.log(np.exp(Z - zmax).sum(1, keepdims=True)))[:, 0]
        lse = own if lse is None else lse
        zk = np.take_along_axis(Z, np.clip(I, 0, vocab - 1).astype(np.int64), 1)
        logp = np.where(P > 0, np.log(np.where(P > 0, P, 1)), 0)
        term = np.where(P > 0, P * (logp - (zk - lse[:, None])), 0)
        size = np.where(P > 0, P * (np.abs(logp) + np.abs(zk) + np.abs(lse)[:, None] + 1), 0)
        q = np.exp(Z - lse[:, None])
        target = np.zeros_like(Z)
        for r in range(rows):
            np.add.at(target[r], np.clip(I[r], 0, vocab - 1), P[r])
        s = np.ones(rows) if scale is None else f64(scale)
        on = live & (s != 0)
        grad = np.where(on[:, None], (q - target) * (s * tau)[:, None], 0)
        gsize = np.where(on[:, None], (q + target) * np.abs(s * tau)[:, None], 0)
    return term.sum(1) * tau * tau, own, grad, size.sum(1) * tau * tau, gsize


def within(got, want, tol, what):
    bad = ~((np.abs(got - want) <= tol) | (got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0], got[bad][:3], want[bad][:3])


def check(ar, z, index, value, scale, tau, dtype, dz=None):
    rows, vocab = z.shape
    loss, lse = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    dz = torch.full_like(z, 7.0) if dz is None else dz
    want_loss, want_lse, want_dz, size, gsize = formula(z, index, value, scale, tau)
    zs = np.abs(f64(z)).max(1) / tau
    ar.check(ar.ar_distill_loss(z, index, value, loss, lse, scale=scale, temperature=tau), "forward")
    alone = (loss.clone(), lse.clone())
    within(f64(lse), want_lse, 2.0 ** -18 * (1 + zs + np.abs(want_lse)), "lse")
    within(f64(loss), want_loss, 2.0 ** -18 * size + 1e-30, "loss")
    tol = U[dtype] * np.abs(want_dz) + 2.0 ** -16 * gsize + TINY[dtype]
    if scale is not None:
        ar.check(ar.ar_distill_loss_backward(z, index, value, lse, scale, dz, temperature=tau), "backward")
        given = formula(z, index, value, scale, tau, f64(lse))
        within(f64(dz), given[2], tol, "dlogits of the backward call")
        dz.fill_(7.0)
    ar.check(ar.ar_distill_loss(z, index, value, loss, lse, scale=scale, dlogits=dz, temperature=tau), "step")
    within(f64(dz), want_dz, tol, "dlogits")
    assert torch.equal(loss, alone[0]) and torch.equal(lse, alone[1])
    return loss, lse, dz


SHAPES = [(1, 1, 1), (2, 3, 3), (3, 8, 2), (5, 1000, 7), (2, 4097, 1), (400, 2049, 16), (6, 50257, 64),
          (1, 131072, 128), (33, 32003, 100), (2, 65536, 1024), (310, 5000, 5)]


@pytest.mark.parametrize("dtype,vdtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"),
                                          ("f16", "f16")])
@pytest.mark.parametrize("rows,vocab,top", SHAPES)
def test_loss_and_gradient(ar, rows, vocab, top, dtype, vdtype):
    z, index, value, scale = make(rows, vocab, top, dtype, 1, vdtype=vdtype)
    check(ar, z, index, value, scale, 2.0, dtype)


@pytest.mark.parametrize("tau", [0.5, 1.0, 3.5])
def test_temperatures_and_no_scale(ar, tau):
    z, index, value, scale = make(9, 3001, 12, "f32", 2)
    check(ar, z, index, value, None, tau, "f32")


@pytest.mark.parametrize("pad,offset,dpad,doffset", [(0, 1, 0, 1), (3, 0, 3, 0), (8, 8, 8, 8), (0, 0, 5, 3), (1, 2, 0, 0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_alignment(ar, dtype, pad, offset, dpad, doffset):
    for rows, vocab in ((7, 5003), (200, 1031), (3, 40000)):
        z, index, value, scale = make(rows, vocab, 9, dtype, 3, pad, offset)
        dz = rows_of(np.zeros((rows, vocab)), dtype, dpad, doffset)
        check(ar, z, index, value, scale, 2.0, dtype, dz)
        if dpad:
            assert torch.isnan(dz._base[doffset:].view(rows, vocab + dpad)[:, vocab:]).all()


def test_lists_that_leave_nothing(ar):
    """Rows without entries, with entries outside the vocabulary, with -inf
    alone, and with scale 0: no loss where there is no distribution, and
    gradients that are exactly zero even where the logits hold NaN."""
    z, index, value, scale = make(8, 4000, 6, "f32", 4)
    index[0] = -1
    index[1, 3:] = 4000
    index[1, :3] = torch.tensor([-5, 2 ** 31 - 1, -2 ** 31], device="cuda")
    value[2] = -float("inf")
    value[3, 1:] = -float("inf")  # one word with probability 1
    scale[4] = 0
    index[5, 2:] = -1
    loss, lse, dz = check(ar, z, index, value, scale, 2.0, "f32")
    assert (loss[:3] == 0).all() and (dz[:3] == 0).all() and (dz[4] == 0).all()
    z[0, 5], z[4, 6] = float("nan"), float("nan")
    ar.check(ar.ar_distill_loss(z, index, value, loss, lse, scale=scale, dlogits=dz, temperature=2.0), "NaN")
    assert (dz[0] == 0).all() and (dz[4] == 0).all() and not torch.isnan(dz).any()
    assert loss[0] == 0 and torch.isnan(lse[0])


def test_no_list_at_all(ar):
    z, _, _, scale = make(4, 500, 1, "bf16", 5)
    empty_i, empty_v = torch.empty(4, 0, dtype=torch.int32, device="cuda"), torch.empty(4, 0, device="cuda")
    loss, lse, dz = check(ar, z, empty_i, empty_v, scale, 1.0, "bf16")
    assert (loss == 0).all() and (dz == 0).all()


def test_infinite_and_large_logits(ar):
    """Words masked with -inf or with the type's lowest value have q = 0; a
    large spread does not overflow."""
    z, index, value, scale = make(4, 3000, 5, "f32", 6)
    z[0, 100:2900] = -float("inf")
    z[1, 1000:] = torch.finfo(torch.float32).min
    z[2] = z[2] * 1e4
    index[:2] = torch.tensor([1, 2, 50, 60, 7], device="cuda")
    index[2] = z[2].topk(5).indices.int()
    loss, lse = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    dz = torch.empty_like(z)
    ar.check(ar.ar_distill_loss(z, index, value, loss, lse, scale=scale, dlogits=dz, temperature=1.0), "masked")
    want_loss, want_lse, want_dz, size, gsize = formula(z, index, value, scale, 1.0)
    assert (dz[0, 100:2900] == 0).all() and (dz[1, 1000:] == 0).all()
    for i, spread in ((0, 1), (1, 1), (2, 2.0 ** 12)):  # exponents of up to 1e5 are off by more units
        within(f64(dz)[i], want_dz[i], 2.0 ** -16 * spread * gsize[i] + 2.0 ** -126, i)
        within(f64(loss)[i:i + 1], want_loss[i:i + 1], 2.0 ** -18 * size[i], i)
    # an entry whose word has q = 0: the loss is infinite, the gradient is not
    index[0, 0] = 500
    ar.check(ar.ar_distill_loss(z, index, value, loss, lse, scale=scale, dlogits=dz, temperature=1.0), "q = 0")
    assert torch.isinf(loss[0]) and torch.isfinite(dz[0]).all() and dz[0, 500] < 0


@pytest.mark.parametrize("rows,vocab,top", [(3, 50257, 40), (500, 1003, 40)])
def test_in_place(ar, rows, vocab, top):
    z, index, value, scale = make(rows, vocab, top, "bf16", 7)
    loss, lse, dz = check(ar, z, index, value, scale, 2.0, "bf16")
    a, b = z.clone(), z.clone()
    l2, s2 = torch.empty_like(loss), torch.empty_like(lse)
    ar.check(ar.ar_distill_loss(a, index, value, l2, s2, scale=scale, dlogits=a, temperature=2.0), "in place")
    ar.check(ar.ar_distill_loss_backward(b, index, value, lse, scale, b, temperature=2.0), "in place")
    assert torch.equal(a, dz) and torch.equal(b, dz) and torch.equal(l2, loss) and torch.equal(s2, lse)


def test_gradient_agrees_with_differences(ar):
    """Central differences of the formula's sum(scale * loss) in 64 bits along
    random directions; their own error at a step of 1e-4 is below 1e-7 of the
    terms."""
    z, index, value, scale = make(5, 300, 8, "f32", 8)
    tau, h = 2.0, 1e-4
    _, _, dz = check(ar, z, index, value, scale, tau, "f32")
    g = np.random.Generator(np.random.PCG64(9))
    for _ in range(6):
        d = torch.from_numpy(g.standard_normal(z.shape)).cuda()
        s = f64(scale)
        up = (formula(z.double() + h * d, index, value, scale, tau)[0] * s).sum()
        down = (formula(z.double() - h * d, index, value, scale, tau)[0] * s).sum()
        want = (f64(dz) * f64(d)).sum()
        assert abs((up - down) / (2 * h) - want) <= 4e-5 * np.abs(f64(dz) * f64(d)).sum()


def test_same_bits_on_another_stream_and_in_a_graph(ar):
    z, index, value, scale = make(40, 20011, 30, "bf16", 10)
    loss, lse, dz = check(ar, z, index, value, scale, 2.0, "bf16")
    out = [torch.empty_like(t) for t in (loss, lse, dz)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ar.check(ar.ar_distill_loss(z, index, value, out[0], out[1], scale=scale, dlogits=out[2], temperature=2.0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, (loss, lse, dz)))


def test_refusals(ar):
    z, index, value, scale = make(4, 100, 5, "bf16", 11)
    loss, lse, dz = torch.empty(4, device="cuda"), torch.empty(4, device="cuda"), torch.empty_like(z)
    bad = ar.AR_ERR_INVALID_ARG
    launches = ar.ar_kernel_launches()
    for tau in (0.0, -1.0, float("nan"), float("inf")):
        assert ar.ar_distill_loss(z, index, value, loss, lse, temperature=tau) == bad
    assert ar.ar_distill_loss(z, index.long(), value, loss, lse) == bad
    assert ar.ar_distill_loss(z, index, value[:, :4], loss, lse) == bad
    assert ar.ar_distill_loss(z, index[:3], value[:3], loss, lse) == bad
    assert ar.ar_distill_loss(z, index, value, loss[:3], lse) == bad
    assert ar.ar_distill_loss(z, index, value, loss, loss) == bad
    assert ar.ar_distill_loss(z, index, value, loss, lse, scale=scale, dlogits=z.t()) == bad
    assert ar.ar_distill_loss(z[:, :50], index, value, loss, lse, dlogits=z[:, 25:75]) == bad
    assert ar.ar_distill_loss(z, index, value, lse, loss, scale=lse) == bad
    assert ar.ar_distill_loss(z, index, value.half(), loss, lse) == ar.AR_ERR_UNSUPPORTED
    assert ar.ar_distill_loss(z.int(), index, value, loss, lse) == ar.AR_ERR_UNSUPPORTED
    assert ar.ar_distill_loss(z.cpu(), index, value, loss, lse) == bad
    wide_i = torch.zeros(4, 1025, dtype=torch.int32, device="cuda")
    assert ar.ar_distill_loss(z, wide_i, wide_i.float(), loss, lse) == -6
    assert ar.ar_distill_loss_backward(z, index, value, lse, lse[:3], dz) == bad
    assert ar.ar_kernel_launches() == launches
    none = torch.empty(0, 100, dtype=torch.bfloat16, device="cuda")
    ar.check(ar.ar_distill_loss(none, index[:0], value[:0], loss[:0], lse[:0]), "no rows")
    assert ar.ar_kernel_launches() == launches


@pytest.mark.parametrize("dtype,vocab,pad,offset", [("bf16", 50257, 0, 0), ("f16", 100003, 5, 3), ("f32", 30001, 0, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_gradient_alone_of_many_long_rows(ar, dtype, vocab, pad, offset, in_place):
    """Rows dealt out in parts: the bits of the call that makes loss and
    gradient, whose first rows are checked against the formula."""
    rows, tau = 310, 1.5
    z, index, value, scale = make(rows, vocab, 20, dtype, 50, pad, offset)
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    want = torch.full_like(z, 7.0)
    ar.check(ar.ar_distill_loss(z, index, value, loss, lse, scale=scale, dlogits=want, temperature=tau), "step")
    n = 3
    exact = formula(z[:n], index[:n], value[:n], scale[:n], tau)
    within(f64(want[:n]), exact[2], U[dtype] * np.abs(exact[2]) + 2.0 ** -16 * exact[4] + TINY[dtype], "dlogits")
    got = z if in_place else torch.full_like(z, 7.0)
    ar.check(ar.ar_distill_loss_backward(z, index, value, lse, scale, got, temperature=tau), "backward")
    assert torch.equal(got, want) and ar.ar_device_status() == (0, 0)
