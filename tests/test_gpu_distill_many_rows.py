"""ar_distill_loss and ar_distill_loss_backward with more rows than four to a
multiprocessor, where blocks take row after row through shared memory, against
the formula in 64 bits (on the device).

Tolerances are those of test_gpu_distill.py, for the same reasons: an exponent
is off by a few binary32 units of |z|/tau + |lse| (below 64 here), a
probability by at most 2^-16 of itself, a loss by 2^-18 of its terms'
magnitudes, lse by 2^-18 of its own.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_distill import DT, TINY, U, ar  # noqa: E402,F401


def many(factor=0.0):
    """A row count past four to a multiprocessor, by the factor."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = max(4 * sms + 1, int(4 * sms * factor))
    assert rows > 4 * sms
    return rows


def make(rows, vocab, top, dtype, seed, pad=0, offset=0, vdtype="f32"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    flat = torch.full((offset + rows * (vocab + pad),), float("nan"), dtype=DT[dtype], device="cuda")
    z = flat[offset:].view(rows, vocab + pad)[:, :vocab]
    z.copy_(torch.randn(rows, vocab, device="cuda", generator=g) * 2)
    index = torch.randint(vocab, (rows, top), device="cuda", generator=g, dtype=torch.int32)  # words may repeat
    value = (torch.randn(rows, top, device="cuda", generator=g) * 2).to(DT[vdtype])
    if top:
        kept = torch.randint(1, top + 1, (rows, 1), device="cuda", generator=g)
        kept[3::7] = 0  # no list
        kept[5::7] = top
        index[torch.arange(top, device="cuda") >= kept] = -1
        index[5, 0], index[12, top - 1] = vocab, 2 ** 31 - 1  # no words
    scale = torch.rand(rows, device="cuda", generator=g) + 0.5
    scale[6::11] = 0
    return z, index, value, scale


def formula(z, index, value, scale, tau, lse=None):
    """loss, lse, dlogits, and the magnitudes of the terms of loss and dlogits, in 64 bits."""
    Z, there = z.double() / tau, (index >= 0) & (index < z.shape[1])
    at = torch.where(there, index, 0).long()
    V = torch.where(there, value.double() / tau, -float("inf"))
    live = there.any(1)
    P = torch.softmax(torch.where(live[:, None], V, 0.0), 1) * there if V.shape[1] else V
    own = torch.logsumexp(Z, 1)
    lse = own if lse is None else lse.double()
    logp, zk = torch.log(torch.where(P > 0, P, 1.0)), torch.gather(Z, 1, at)
    loss = (P * (logp - zk + lse[:, None])).sum(1) * tau * tau
    size = (P * (logp.abs() + zk.abs() + lse.abs()[:, None] + 1)).sum(1) * tau * tau
    s = (torch.ones_like(own) if scale is None else scale.double()) * tau
    on = (live & (s != 0))[:, None]
    Z.sub_(lse[:, None]).exp_()
    target = torch.zeros_like(Z).scatter_add_(1, at, P)
    grad = torch.where(on, (Z - target) * s[:, None], 0.0)
    gsize = torch.where(on, Z.add_(target) * s.abs()[:, None], 0.0)
    return loss, own, grad, size, gsize


def within(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][:3].tolist(), want[bad][:3].tolist())


def check(ar, z, index, value, scale, tau, dtype, into=None):
    """All three forms of the call: loss alone, loss and gradient, gradient alone."""
    rows, vocab = z.shape
    loss, lse = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    dz = torch.full(z.shape, 7.0, dtype=z.dtype, device="cuda") if into is None else into
    zs = z.abs().amax(1).double() / tau
    ar.check(ar.ar_distill_loss(z, index, value, loss, lse, scale=scale, temperature=tau), "loss")
    alone = loss.clone(), lse.clone()
    want_loss, want_lse, want, size, gsize = formula(z, index, value, scale, tau)
    within(lse, want_lse, 2.0 ** -18 * (1 + zs + want_lse.abs()), "lse")
    within(loss, want_loss, 2.0 ** -18 * size + 1e-30, "loss")
    ar.check(ar.ar_distill_loss(z, index, value, loss, lse, scale=scale, dlogits=dz, temperature=tau), "step")
    assert torch.equal(loss, alone[0]) and torch.equal(lse, alone[1])
    within(dz, want, U[dtype] * want.abs() + 2.0 ** -16 * gsize + TINY[dtype], "dlogits of the step")
    step = dz.clone()
    if scale is not None:
        dz.fill_(7.0)
        ar.check(ar.ar_distill_loss_backward(z, index, value, lse, scale, dz, temperature=tau), "backward")
        assert torch.equal(dz, step)  # the lse is the same, so the bits are
    assert ar.ar_device_status() == (0, 0)
    return loss, lse, step


# Rows of one piece, of several, of as many as shared memory keeps for the
# second pass, and of more (copied in twice); the gradient alone by whole rows,
# halves (8 pieces of 12288 bytes) and quarters (16 of them).
@pytest.mark.parametrize("dtype,vdtype,vocab,top", [
    ("bf16", "f32", 1, 1), ("f16", "f16", 5, 3), ("bf16", "bf16", 1003, 40), ("f32", "f32", 6144, 7),
    ("bf16", "f32", 6144, 1), ("f16", "f32", 6145, 33), ("f32", "f32", 20011, 64), ("bf16", "f32", 50257, 64),
    ("bf16", "f32", 50257, 128), ("f16", "f16", 100003, 20), ("bf16", "bf16", 120001, 16), ("f32", "f32", 43501, 1024),
    ("f32", "f32", 60013, 100), ("f16", "f32", 2048, 1024)])
def test_loss_and_gradient(ar, dtype, vdtype, vocab, top):
    z, index, value, scale = make(many(), vocab, top, dtype, 1, vdtype=vdtype)
    check(ar, z, index, value, scale, 2.0, dtype)


@pytest.mark.parametrize("factor", [1.7, 3.3])
@pytest.mark.parametrize("dtype,vocab", [("f32", 5003), ("bf16", 30001)])
def test_several_rows_to_a_block(ar, dtype, vocab, factor):
    z, index, value, scale = make(many(factor), vocab, 9, dtype, 2)
    check(ar, z, index, value, scale, 1.5, dtype)


def test_so_many_rows_that_places_are_used_again_and_again(ar):
    z, index, value, scale = make(20000, 700, 5, "bf16", 3)
    check(ar, z, index, value, scale, 1.0, "bf16")
    z, index, value, scale = make(20000, 700, 5, "f32", 4)
    check(ar, z, index, value, None, 1.0, "f32")


@pytest.mark.parametrize("pad,offset,dpad,doffset", [(0, 1, 0, 1), (3, 0, 3, 0), (8, 8, 8, 8), (0, 0, 5, 3), (1, 2, 0, 0)])
@pytest.mark.parametrize("dtype,vocab", [("f32", 3073), ("bf16", 1031), ("f16", 24583), ("bf16", 98304)])
def test_strides_and_alignment(ar, dtype, vocab, pad, offset, dpad, doffset):
    rows = many()
    z, index, value, scale = make(rows, vocab, 9, dtype, 5, pad, offset)
    flat = torch.full((doffset + rows * (vocab + dpad),), float("nan"), dtype=DT[dtype], device="cuda")
    check(ar, z, index, value, scale, 2.0, dtype, flat[doffset:].view(rows, vocab + dpad)[:, :vocab])
    if dpad:
        assert torch.isnan(flat[doffset:].view(rows, vocab + dpad)[:, vocab:]).all()
    assert torch.isnan(flat[:doffset]).all()


@pytest.mark.parametrize("dtype,vocab,top,pad,offset", [
    ("bf16", 1003, 40, 0, 0), ("bf16", 50257, 40, 0, 0), ("bf16", 50257, 40, 3, 1), ("f16", 100003, 20, 0, 0),
    ("f32", 43501, 1024, 0, 3), ("f32", 60013, 20, 5, 0), ("bf16", 120001, 16, 0, 0)])
def test_in_place(ar, dtype, vocab, top, pad, offset):
    z, index, value, scale = make(many(1.3), vocab, top, dtype, 6, pad, offset)
    loss, lse, dz = check(ar, z, index, value, scale, 2.0, dtype)
    kept = z.clone()
    l2, s2 = torch.empty_like(loss), torch.empty_like(lse)
    ar.check(ar.ar_distill_loss(z, index, value, l2, s2, scale=scale, dlogits=z, temperature=2.0), "in place")
    assert torch.equal(z, dz) and torch.equal(l2, loss) and torch.equal(s2, lse)
    z.copy_(kept)
    ar.check(ar.ar_distill_loss_backward(z, index, value, lse, scale, z, temperature=2.0), "in place")
    assert torch.equal(z, dz)


def test_no_list_at_all(ar):
    z, index, value, scale = make(many(), 5003, 0, "bf16", 7)
    loss, lse, dz = check(ar, z, index, value, scale, 1.0, "bf16")
    assert (loss == 0).all() and (dz == 0).all()


def test_masked_words(ar):
    """Words of -inf or of the type's lowest value have q = 0."""
    z, index, value, scale = make(many(), 4099, 8, "f32", 8)
    z[:, 2000:3000] = -float("inf")
    z[1::2, 3500:] = torch.finfo(torch.float32).min
    index.clamp_(max=1999)
    loss, lse = torch.empty(len(z), device="cuda"), torch.empty(len(z), device="cuda")
    dz = torch.empty_like(z)
    ar.check(ar.ar_distill_loss(z, index, value, loss, lse, scale=scale, dlogits=dz), "masked")
    want_loss, want_lse, want, size, gsize = formula(z, index, value, scale, 1.0)
    within(lse, want_lse, 2.0 ** -18 * (16 + want_lse.abs()), "lse")
    within(loss, want_loss, 2.0 ** -18 * size + 1e-30, "loss")
    within(dz, want, U["f32"] * want.abs() + 2.0 ** -16 * gsize + TINY["f32"], "dlogits")
    assert (dz[:, 2000:3000] == 0).all()


def test_same_bits_on_another_stream_and_in_a_graph(ar):
    z, index, value, scale = make(many(1.7), 20011, 30, "bf16", 9)
    loss, lse, dz = check(ar, z, index, value, scale, 2.0, "bf16")
    out = [torch.empty_like(t) for t in (loss, lse, dz)]
    back = torch.empty_like(dz)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ar.check(ar.ar_distill_loss(z, index, value, out[0], out[1], scale=scale, dlogits=out[2], temperature=2.0))
        ar.check(ar.ar_distill_loss_backward(z, index, value, out[1], scale, back, temperature=2.0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out + [back], (loss, lse, dz, dz)))
