"""ar_diff_attention and ar_diff_attention_backward against the formulas in 64
bits.

Tolerances.  u is the tensors' unit roundoff (2^-8 bf16, 2^-11 f16).  A result is
rounded once (u of itself), and so is every probability, difference of
probabilities or ds before the product that sums it: u of the sum of the terms'
magnitudes.  Scores, and the products dout.v, dout.out and dout.second, are
binary32 sums of exact products of at most 128 terms: off by at most 2^-17 of the
sum of the terms' magnitudes, which enters a probability as a relative error; the
exponential adds a few units of its exponent, which stays below 2^-13 here.
Probabilities below the smallest normal number of f16 are off by 2^-25 of the
row's largest, and so are results there (half of f16's spacing).  dlambda is a
binary32 sum of at most 2200 terms, 7 in a thread, then 15 levels, each of which
is off as above: 2^-16 of the sum of magnitudes.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LOST = {"bf16": 0.0, "f16": 2.0 ** -25}
SCORE = 2.0 ** -17
EXP = 2.0 ** -13


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


def packed(lengths, before=0):
    return torch.tensor(np.cumsum([before] + list(lengths)), dtype=torch.int32, device="cuda")


def make(tokens, heads, kv, dim, vdim, dtype, seed, lam=None):
    """q, k, v, lambda and dout"""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q, k, v, dout = (torch.randn(tokens, *s, device="cuda", generator=g).to(DT[dtype]) for s in (
        (2 * heads, dim), (2 * kv, dim), (kv, vdim), (heads, vdim)))
    if lam is None:
        lam = torch.rand(heads, device="cuda", generator=g)
    else:
        lam = torch.tensor([lam[i % len(lam)] for i in range(heads)], device="cuda")
    return q, k, v, lam, dout


def sequences(cu):
    c = cu.tolist()
    return [(a, b) for a, b in zip(c, c[1:]) if b > a]


def covered(cu, tokens):
    c = np.zeros(tokens, bool)
    for a, b in sequences(cu):
        c[a:b] = True
    return c


def reference(q, k, v, lam, cu, scale, dout=None, out=None, second=None, lse=None):
    """Results (out, second, lse; or dq, dk, dv, dlam) and name + "_tol", what
    their roundings before the last and the arithmetic may cost, in parts: _u
    (times u), _off, and _all (times LOST)."""
    t, h, kv, d, e = q.shape[0], lam.shape[0], v.shape[1], q.shape[2], v.shape[2]
    group, L = h // kv, f64(lam)
    shapes = {"out": (t, h, e), "second": (t, h, e), "lse": (t, 2 * h), "dq": q.shape, "dk": k.shape, "dv": v.shape, "dlam": (h,)}
    r = {n + s: np.zeros(x) for n, x in shapes.items() for s in ("", "_u", "_off", "_all")}

    def put(name, at, value, u, off, all_):
        for s, x in zip(("", "_u", "_off", "_all"), (value, u, off, all_)):
            r[name + s][at] += x

    for a, b in sequences(cu):
        n = b - a
        mask = np.triu(np.ones((n, n), bool), 1)
        for j in range(h):
            i = j // group
            V, lj = f64(v[a:b, i]), L[j]
            p, rel, Q, K = [], [], [], []
            for m in (0, 1):
                Q.append(f64(q[a:b, 2 * j + m]))
                K.append(f64(k[a:b, 2 * i + m]))
                s = Q[m] @ K[m].T * scale
                s[mask] = -np.inf
                size = (np.abs(Q[m]) @ np.abs(K[m]).T * scale * ~mask).max(1)
                rel.append(EXP + SCORE * size[:, None])
                if dout is None:
                    top = s.max(1, keepdims=True)
                    x = np.exp(s - top)
                    p.append(x / x.sum(1, keepdims=True))
                    full = (top + np.log(x.sum(1, keepdims=True)))[:, 0]
                    put("lse", (slice(a, b), 2 * j + m), full, 0, SCORE * size + 2.0 ** -18 * (1 + np.abs(full)), 0)
                else:
                    p.append(np.exp(s - f64(lse[2 * j + m, a:b])[:, None]))
            at, kat = (slice(a, b), j), (slice(a, b), i)
            aV, seen = np.abs(V), ~mask
            if dout is None:
                w = [x @ aV for x in p]
                put("second", at, p[1] @ V, w[1], rel[1] * w[1], 1 + seen @ aV)
                put("out", at, (p[0] - lj * p[1]) @ V, w[0] + abs(lj) * w[1], rel[0] * w[0] + abs(lj) * rel[1] * w[1],
                    (1 + abs(lj)) * (1 + seen @ aV))
                continue
            DO, O, S = f64(dout[a:b, j]), f64(out[a:b, j]), f64(second[a:b, j])
            aD = np.abs(DO)
            dp, dp_size = DO @ V.T, aD @ aV.T
            delta = [(DO * O).sum(1) + lj * (DO * S).sum(1), (DO * S).sum(1)]
            delta_size = [(aD * np.abs(O)).sum(1) + abs(lj) * (aD * np.abs(S)).sum(1), (aD * np.abs(S)).sum(1)]
            c = p[0] - lj * p[1]
            put("dv", kat, c.T @ DO, np.abs(c).T @ aD, (p[0] * rel[0] + abs(lj) * p[1] * rel[1]).T @ aD,
                (1 + abs(lj)) * (1 + seen.T @ aD))
            put("dlam", j, -delta[1].sum(), 0, 2.0 ** -16 * delta_size[1].sum(), 0)
            for m, f in ((0, 1.0), (1, -lj)):
                ds = p[m] * (dp - delta[m][:, None])
                off = np.abs(ds) * rel[m] + p[m] * SCORE * (dp_size + delta_size[m][:, None])
                for name, x, y, where in (("dq", ds, K[m], (slice(a, b), 2 * j + m)), ("dk", ds.T, Q[m], (slice(a, b), 2 * i + m))):
                    o, sn = (off, seen) if name == "dq" else (off.T, seen.T)
                    put(name, where, f * scale * x @ y, abs(f) * scale * np.abs(x) @ np.abs(y), abs(f) * scale * o @ np.abs(y),
                        (1 + abs(f)) * (1 + scale * sn @ np.abs(y)))
    return r


def check(ar, q, k, v, lam, cu, dtype, dout=None, scale=None, outs=None, grads=None):
    t, h, kv, d, e = q.shape[0], lam.shape[0], v.shape[1], q.shape[2], v.shape[2]
    s = d ** -0.5 if scale is None else scale
    if outs is None:
        outs = [torch.full((t, h, e), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    out, second = outs
    lse = torch.full((2 * h, t), 7.0, device="cuda")
    ar.check(ar.ar_diff_attention(q, k, v, lam, cu, out, second, lse, scale=scale), "ar_diff_attention")
    assert ar.ar_device_status() == (0, 0)
    r, on = reference(q, k, v, lam, cu, s), covered(cu, t)

    def compare(name, x, twice=1):
        tol = U[dtype] * (np.abs(r[name]) + r[name + "_u"] * (1 + EXP)) + twice * r[name + "_off"] + LOST[dtype] * r[name + "_all"]
        within(x[on], r[name][on], tol[on], name)
        assert (x[~on] == 7).all()  # tokens of no sequence

    compare("out", f64(out))
    compare("second", f64(second))
    within(f64(lse).T[on], r["lse"][on], r["lse_off"][on], "lse")
    assert (f64(lse).T[~on] == 7).all()
    if dout is None:
        return out, second, lse
    if grads is None:
        grads = [torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda") for x in (q, k, v)]
    dlam = torch.full((h,), 7.0, device="cuda")
    ws = torch.full((ar.ar_diff_attention_workspace_bytes(t, h, kv, d, e),), 0xFF, dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_diff_attention_backward(dout, q, k, v, lam, out, second, lse, cu, *grads, dlam, ws, scale=scale),
             "ar_diff_attention_backward")
    assert ar.ar_device_status() == (0, 0)
    r = reference(q, k, v, lam, cu, s, dout, out, second, lse)
    for x, name in zip(grads, ("dq", "dk", "dv")):
        compare(name, f64(x), 2)
    within(f64(dlam), r["dlam"], r["dlam_off"] + 1e-30, "dlam")
    return out, second, lse, grads, dlam


LENGTHS = [[1], [2], [63], [64], [65], [127], [128], [129], [192], [255], [256], [257], [300, 1, 0, 77, 128], [1, 1, 1],
           [513], [64, 640]]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,vdim", [(64, 128), (32, 64)])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_lengths(ar, lengths, dim, vdim, dtype):
    *x, dout = make(sum(lengths), 2, 1, dim, vdim, dtype, 1)
    check(ar, *x, packed(lengths), dtype, dout)


@pytest.mark.parametrize("dim,vdim", [(8, 8), (8, 128), (16, 16), (24, 48), (40, 80), (48, 96), (56, 72), (64, 8), (64, 64),
                                      (64, 104), (64, 120)])
def test_head_sizes(ar, dim, vdim):
    *x, dout = make(200, 3, 3, dim, vdim, "bf16", 2)
    check(ar, *x, packed([150, 50]), "bf16", dout)


@pytest.mark.parametrize("heads,kv", [(1, 1), (6, 6), (8, 2), (6, 1), (16, 4)])
def test_shared_heads(ar, heads, kv):
    *x, dout = make(290, heads, kv, 64, 128, "f16", 3)
    check(ar, *x, packed([131, 159]), "f16", dout)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lam", [(0.0,), (1.0,), (-0.7, 0.3), (2.5,), (-40.0, 0.01), (1e-6,), (1e-6, 0.8), (0.0, 0.5)])
def test_lambda(ar, dtype, lam):
    """Any size and sign; heads of a group that differ by many powers of two."""
    *x, dout = make(270, 4, 2, 64, 128, dtype, 4, lam)
    check(ar, *x, packed([200, 70]), dtype, dout)


def test_lambda_of_zero_is_the_first_map(ar):
    q, k, v, lam, dout = make(150, 2, 2, 64, 64, "bf16", 5, (0.0,))
    out, second, lse, grads, dlam = check(ar, q, k, v, lam, packed([150]), "bf16", dout)
    plain, plain_lse = torch.empty_like(out), torch.empty(2, 150, device="cuda")
    first = [t[:, ::2].contiguous() for t in (q, k)]
    ar.check(ar.ar_attention(*first, v, packed([150]), plain, plain_lse), "ar_attention")
    assert (out.float() - plain.float()).abs().max() <= 2.0 ** -7 * plain.abs().max()
    assert (grads[0][:, 1::2] == 0).all() and (grads[1][:, 1::2] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lam", [(1e-40,), (-1e-45, 0.0), (1.4e-39, -2.9e-39)])
def test_a_lambda_whose_reciprocal_is_no_number(ar, dtype, lam):
    """Gradients of the second map are below 1e-37, all others those without it.
    (bf16 has multiples of 2^-133 there, 9e-41: nothing relative is asked.)"""
    *x, no, dout = make(150, 4, 2, 64, 64, dtype, 24, (0.0,))
    cu, few = packed([100, 50]), torch.tensor([lam[i % len(lam)] for i in range(4)], device="cuda")
    *want, (dq, dk, dv), dlam = check(ar, *x, no, cu, dtype, dout)
    got, g, got_dlam = [torch.empty_like(t) for t in want], [torch.empty_like(t) for t in x], torch.empty(4, device="cuda")
    ws = torch.empty(ar.ar_diff_attention_workspace_bytes(150, 4, 2, 64, 64), dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_diff_attention(*x, few, cu, *got), "forward")
    ar.check(ar.ar_diff_attention_backward(dout, *x, few, *got, cu, *g, got_dlam, ws), "backward")
    for a, b in ((dq, g[0]), (dk, g[1])):
        assert torch.equal(a[:, ::2], b[:, ::2]) and b[:, 1::2].abs().max() <= 1e-37
    for a, b in zip((*want, dv, dlam), (*got, g[2], got_dlam)):
        assert torch.equal(a, b)


def test_many_sequences(ar):
    """More sequences than a warp looks at at once, empty ones among them."""
    g = np.random.Generator(np.random.PCG64(6))
    lengths = [int(x) for x in g.integers(0, 40, 150)]
    lengths[70] = 400
    *x, dout = make(sum(lengths), 2, 2, 64, 128, "bf16", 7)
    check(ar, *x, packed(lengths), "bf16", dout)


def test_long_sequence(ar):
    *x, dout = make(2111, 2, 1, 64, 128, "bf16", 8)
    check(ar, *x, packed([2111]), "bf16", dout)


def test_growing_scores(ar):
    """Keys that grow along the sequence, the second map's faster, so that rows'
    maxima keep moving and outputs are rescaled again and again."""
    q, k, v, lam, dout = make(1100, 2, 2, 64, 128, "f16", 9)
    q = q.abs() * 0.5
    rise = torch.arange(1100, device="cuda")[:, None, None] / 250
    k = (k.abs() * 0.25 + rise * torch.tensor([1.0, 1.5, 1.0, 1.5], device="cuda")[:, None]).to(k.dtype)
    check(ar, q, k, v, lam, packed([1100]), "f16", dout)


def test_scale(ar):
    *x, dout = make(140, 2, 2, 64, 128, "bf16", 10)
    for scale in (0.02, 0.5):
        check(ar, *x, packed([140]), "bf16", dout, scale=scale)


@pytest.mark.parametrize("power", [-20, -13, 9, 13])
def test_f16_gradients_of_any_size(ar, power):
    """Upstream gradients times powers of two: what f16 cannot hold as it is is
    held times another power.  A gradient that is a number of f16 is as exact as
    ever; below its smallest normal number spacings are 2^-24."""
    q, k, v, lam, dout = make(300, 2, 1, 64, 128, "f16", 11)
    v = v * (0.25 if power > 9 else 1)
    check(ar, q, k, v, lam, packed([170, 130]), "f16", (dout.float() * 2.0 ** power).half())


def test_tokens_outside_every_sequence(ar):
    """They are neither read (they hold NaN) nor written, and no part of dlambda."""
    q, k, v, lam, dout = make(500, 2, 1, 64, 128, "bf16", 12)
    for lengths, before in (([200, 130], 37), ([0, 0], 3)):
        cu = packed(lengths, before)
        off = torch.from_numpy(~covered(cu, 500)).cuda()
        x = [t.clone() for t in (q, k, v, dout)]
        for t in x:
            t[off] = float("nan")
        check(ar, *x[:3], lam, cu, "bf16", x[3])


@pytest.mark.parametrize("layout", ["one projection", "heads outside", "padded", "maps apart"])
def test_layouts(ar, layout):
    t, h, kv, d, e, dtype = 333, 4, 2, 64, 128, "bf16"
    q0, k0, v0, lam, dout0 = make(t, h, kv, d, e, dtype, 13)

    def place(*parts):
        if layout == "one projection" and len({p.shape[2] for p in parts}) == 1:
            whole = torch.cat(parts, 1).contiguous()
            return list(torch.split(whole, [p.shape[1] for p in parts], 1))
        if layout == "heads outside":
            return [p.transpose(0, 1).contiguous().transpose(0, 1) for p in parts]
        if layout == "padded":
            return [torch.nn.functional.pad(p, (0, 24, 0, 1))[:, :-1, :p.shape[2]] for p in parts]
        if layout == "maps apart":
            return [torch.stack([p, torch.zeros_like(p)], 2)[:, :, 0] for p in parts]
        return [p.contiguous() for p in parts]

    def seven(x):
        return torch.full_like(x, 7.0)

    (q, k), (v,), (dout,) = place(q0, k0), place(v0), place(dout0)
    outs = place(seven(dout0)) + place(seven(dout0))
    grads = place(seven(q0), seven(k0)) + place(seven(v0))
    check(ar, q, k, v, lam, packed([200, 133]), dtype, dout, outs=outs, grads=grads)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_other_sequences_do_not_matter(ar, bad, dtype):
    """Every tensor of the middle sequence is not finite: the others' results
    keep their bits."""
    t, lengths = 570, [130, 250, 190]
    q, k, v, lam, dout = make(t, 2, 1, 64, 128, dtype, 14)
    cu = packed(lengths)
    clean = check(ar, q, k, v, lam, cu, dtype, dout)
    results = [clean[0], clean[1], clean[2].t(), *clean[3]]
    x = [a.clone() for a in (q, k, v, dout)]
    for a in x:
        a[130:380] = bad
    out, second = torch.empty_like(dout), torch.empty_like(dout)
    lse, grads, dlam = torch.empty(4, t, device="cuda"), [torch.empty_like(a) for a in (q, k, v)], torch.empty(2, device="cuda")
    ws = torch.empty(ar.ar_diff_attention_workspace_bytes(t, 2, 1, 64, 128), dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_diff_attention(*x[:3], lam, cu, out, second, lse), "forward")
    ar.check(ar.ar_diff_attention_backward(x[3], *x[:3], lam, out, second, lse, cu, *grads, dlam, ws), "backward")
    for a, b in zip(results, (out, second, lse.t(), *grads)):
        for at in (slice(0, 130), slice(380, 570)):
            assert torch.equal(a[at], b[at])
    assert torch.isnan(dlam).all() and ar.ar_device_status() == (0, 0)


def test_later_keys_do_not_matter(ar):
    """Scores of later tokens may be anything; values that are not finite reach
    no token more than 127 before their own."""
    q, k, v, lam, _ = make(400, 2, 1, 64, 128, "bf16", 15)
    cu = packed([400])
    out, second, lse = check(ar, q, k, v, lam, cu, "bf16")
    k2, v2 = k.clone(), v.clone()
    k2[300:] = float("nan")
    v2[390:] = float("inf")
    got, got2, got_lse = torch.empty_like(out), torch.empty_like(out), torch.empty_like(lse)
    ar.check(ar.ar_diff_attention(q, k2, v2, lam, cu, got, got2, got_lse), "forward")
    assert torch.equal(got[:263], out[:263]) and torch.equal(got2[:263], second[:263])
    assert torch.equal(got_lse[:, :300], lse[:, :300]) and torch.isnan(got[300:]).all()


@pytest.mark.parametrize("tokens", [100, 300, 449])
def test_a_key_of_minus_infinity(ar, tokens):
    """A key whose scores are all -inf in the second map has no weight there: it
    gets a zero gradient from that map, all others finite ones."""
    q, k, v, lam, dout = make(tokens, 2, 1, 64, 128, "bf16", 16)
    q[:, 1::2, 0] = q[:, 1::2, 0].abs() + 0.5
    k[5, 1, 0] = -float("inf")
    cu = packed([tokens])
    out, second, lse = torch.empty_like(dout), torch.empty_like(dout), torch.empty(4, tokens, device="cuda")
    dq, dk, dv, dlam = (torch.full_like(x, 7.0) for x in (q, k, v, lam))
    ws = torch.empty(ar.ar_diff_attention_workspace_bytes(tokens, 2, 1, 64, 128), dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_diff_attention(q, k, v, lam, cu, out, second, lse), "forward")
    ar.check(ar.ar_diff_attention_backward(dout, q, k, v, lam, out, second, lse, cu, dq, dk, dv, dlam, ws), "backward")
    assert torch.isfinite(out).all() and torch.isfinite(second).all() and torch.isfinite(lse).all()
    assert (dk[5, 1] == 0).all() and torch.isfinite(dk).all() and torch.isfinite(dv).all() and torch.isfinite(dlam).all()
    assert torch.isfinite(dq[:, :, 1:]).all() and torch.isfinite(dq[:, ::2]).all()


def test_first_token_sees_itself_alone(ar):
    q, k, v, lam, _ = make(50, 2, 2, 64, 64, "f16", 17)
    out, second, _ = check(ar, q, k, v, lam, packed([1, 30, 19]), "f16")
    for first in (0, 1, 31):
        assert torch.equal(second[first], v[first])


def test_gradient_agrees_with_differences(ar):
    """All four gradients against central differences of the formula's sum(out *
    dout) in 64 bits: at a step of 1e-4 their own error is below 1e-6 of the
    terms; the gradients' is at most u twice, for each of their terms, and what
    out and second, which deltas are made of, are off by themselves."""
    lengths, scale, h = [5, 9], 0.3, 1e-4
    q, k, v, lam, dout = make(14, 4, 2, 16, 24, "f16", 18)
    cu = packed(lengths)
    *_, grads, dlam = check(ar, q, k, v, lam, cu, "f16", dout, scale=scale)

    def total(*x):
        return (reference(*x, cu, scale)["out"] * f64(dout)).sum()

    g = torch.Generator(device="cuda")
    g.manual_seed(19)
    base = [x.double() for x in (q, k, v, lam)]
    for _ in range(6):
        d = [torch.randn(x.shape, device="cuda", generator=g, dtype=torch.float64) for x in base]
        up = total(*(x + h * e for x, e in zip(base, d)))
        down = total(*(x - h * e for x, e in zip(base, d)))
        terms = [x.double() * e for x, e in zip((*grads, dlam), d)]
        got, size = sum(x.sum().item() for x in terms), sum(x.abs().sum().item() for x in terms)
        assert abs((up - down) / (2 * h) - got) <= 6 * U["f16"] * size


def test_same_bits_call_after_call_on_a_full_device(ar):
    """More blocks than the device holds, again and again: sums are made in one
    order, and no warp is a step ahead of a barrier."""
    for dtype in ("bf16", "f16"):
        q, k, v, lam, dout = make(3000, 6, 2, 64, 128, dtype, 20)
        cu = packed([1000, 7, 400, 1593])
        t, first = 3000, None
        for _ in range(25):
            out, second, lse = torch.empty_like(dout), torch.empty_like(dout), torch.empty(12, t, device="cuda")
            grads, dlam = [torch.empty_like(x) for x in (q, k, v)], torch.empty(6, device="cuda")
            ws = torch.empty(ar.ar_diff_attention_workspace_bytes(t, 6, 2, 64, 128), dtype=torch.uint8, device="cuda")
            ar.check(ar.ar_diff_attention(q, k, v, lam, cu, out, second, lse), "forward")
            ar.check(ar.ar_diff_attention_backward(dout, q, k, v, lam, out, second, lse, cu, *grads, dlam, ws), "backward")
            now = [out, second, lse, *grads, dlam]
            first = first or now
            assert all(torch.equal(a, b) for a, b in zip(now, first))
        assert ar.ar_device_status() == (0, 0)


def test_same_bits_on_another_stream_and_in_graphs(ar):
    """Also two graphs that share a workspace, replayed one after the other."""
    t = 600
    q, k, v, lam, dout = make(t, 4, 2, 64, 128, "bf16", 21)
    cu = packed([250, 350])
    out, second, lse, grads, dlam = check(ar, q, k, v, lam, cu, "bf16", dout)
    want2 = check(ar, q, k, v, lam, cu, "bf16", dout * 2)
    ws = torch.empty(ar.ar_diff_attention_workspace_bytes(t, 4, 2, 64, 128), dtype=torch.uint8, device="cuda")
    got, graphs = [], []
    for up in (dout, dout * 2):
        to = [torch.zeros_like(x) for x in (out, second, lse, *grads, dlam)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ar.check(ar.ar_diff_attention(q, k, v, lam, cu, *to[:3]), "forward")
            ar.check(ar.ar_diff_attention_backward(up, q, k, v, lam, *to[:3], cu, *to[3:], ws), "backward")
        got.append(to)
        graphs.append((graph, up))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for x in got[0] + got[1]:
            x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for graph, _ in graphs:
                graph.replay()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[0], (out, second, lse, *grads, dlam)))
        assert all(torch.equal(a, b) for a, b in zip(got[1], (*want2[:3], *want2[3], want2[4])))


def test_what_may_be_left_out(ar):
    q, k, v, lam, dout = make(170, 2, 2, 64, 128, "bf16", 22)
    cu = packed([170])
    out, second, lse, grads, dlam = check(ar, q, k, v, lam, cu, "bf16", dout)
    got = torch.empty_like(out)
    ar.check(ar.ar_diff_attention(q, k, v, lam, cu, got), "neither second nor lse")
    assert torch.equal(got, out)
    g2 = [torch.empty_like(x) for x in grads]
    ws = torch.empty(ar.ar_diff_attention_workspace_bytes(170, 2, 2, 64, 128), dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_diff_attention_backward(dout, q, k, v, lam, out, second, lse, cu, *g2, None, ws), "no dlambda")
    assert all(torch.equal(a, b) for a, b in zip(g2, grads))


def test_lengths_that_are_not_sound_stay_inside_the_tensors(ar):
    """Entries outside [0, tokens] are clamped, a decreasing pair is an empty
    sequence."""
    q, k, v, lam, dout = make(100, 2, 2, 64, 128, "bf16", 23)
    whole = check(ar, q, k, v, lam, packed([100]), "bf16", dout)
    for entries, same in (([-5, 1000], True), ([60, 20], False)):
        cu = torch.tensor(entries, dtype=torch.int32, device="cuda")
        out, second, lse = torch.zeros_like(dout), torch.zeros_like(dout), torch.zeros(4, 100, device="cuda")
        grads, dlam = [torch.zeros_like(x) for x in (q, k, v)], torch.empty(2, device="cuda")
        ws = torch.empty(ar.ar_diff_attention_workspace_bytes(100, 2, 2, 64, 128), dtype=torch.uint8, device="cuda")
        ar.check(ar.ar_diff_attention(q, k, v, lam, cu, out, second, lse), "forward")
        ar.check(ar.ar_diff_attention_backward(dout, q, k, v, lam, out, second, lse, cu, *grads, dlam, ws), "backward")
        got = [out, second, lse, *grads, dlam]
        if same:
            assert all(torch.equal(a, b) for a, b in zip(got, (*whole[:3], *whole[3], whole[4])))
        else:
            assert all((x == 0).all() for x in got)
    assert ar.ar_device_status() == (0, 0)


def test_refusals(ar):
    q, k, v, lam, dout = make(40, 4, 2, 64, 128, "bf16", 24)
    out, second, lse, cu = torch.empty_like(dout), torch.empty_like(dout), torch.empty(8, 40, device="cuda"), packed([40])
    bad, unsupported, call = ar.AR_ERR_INVALID_ARG, ar.AR_ERR_UNSUPPORTED, ar.ar_diff_attention
    launches = ar.ar_kernel_launches()
    f = [x.float() for x in (q, k, v)]
    assert call(*f, lam, cu, out.float(), second.float(), lse) == unsupported
    assert call(q, k.half(), v, lam, cu, out, second, lse) == bad
    assert call(q, k[:, :, :32], v, lam, cu, out, second, lse) == bad
    assert call(q, k[:, :2], v, lam, cu, out, second, lse) == bad                    # one map's keys alone
    assert call(q[:, :4], k, v, lam, cu, out, second, lse) == bad
    assert call(q[:, :6], k, v, lam[:3], cu, out[:, :3], second[:, :3], lse[:6]) == bad  # 3 heads over 2
    assert call(q, k, v, lam.double(), cu, out, second, lse) == bad and call(q, k, v, lam[:, None], cu, out, second, lse) == bad
    assert call(q, k, v, lam, cu.long(), out, second, lse) == bad and call(q, k, v, lam, cu.cpu(), out, second, lse) == bad
    assert call(q, k, v, lam.cpu(), cu, out, second, lse) == bad
    assert call(q, k, v, lam, cu, out[:39], second, lse) == bad and call(q, k, v, lam, cu, out, second, lse[:4]) == bad
    assert call(q, k, v, lam, cu, out[..., :64], second, lse) == bad
    assert call(q, k, v, lam, cu, out, out, lse) == bad and call(q, k, v, lam, cu, dout, v.repeat(1, 2, 1), lse.half()) == bad
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(q, k, v, lam, cu, out, second, lse, scale=scale) == bad
    wide = torch.zeros(40, 8, 72, dtype=torch.bfloat16, device="cuda")
    assert call(wide, wide[:, :4], v, lam, cu, out, second, lse) == unsupported       # heads of 72
    assert call(wide[:, :, 1:65], k, v, lam, cu, out, second, lse) == bad
    odd = torch.zeros(40, 2, 100, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(40, 4, 100, dtype=torch.bfloat16, device="cuda")
    assert call(q, k, odd, lam, cu, o, o.clone(), lse) == unsupported
    dq, dk, dv, dlam = (torch.empty_like(x) for x in (q, k, v, lam))
    ws = torch.empty(ar.ar_diff_attention_workspace_bytes(40, 4, 2, 64, 128), dtype=torch.uint8, device="cuda")
    back = ar.ar_diff_attention_backward
    args = (dout, q, k, v, lam, out, second, lse, cu)
    assert back(*args, dq, dk, dv, dlam, ws[:-1]) == bad and back(*args, dq, dk, dv, dlam[:3], ws) == bad
    assert back(*args, q, dk, dv, dlam, ws) == bad and back(*args, dq, dk, dv, lam, ws) == bad
    assert back(dout, q, k, v, lam, out, second, None, cu, dq, dk, dv, dlam, ws) == bad
    assert ar.ar_kernel_launches() == launches
    none = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    nv, no = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    assert call(none, none[:, :4], nv, lam, cu, no) == ar.AR_OK
    assert call(q, k, v, lam, cu[:1], out, second, lse) == ar.AR_OK
    dlam.fill_(7)
    assert back(dout, q, k, v, lam, out, second, lse, cu[:1], dq, dk, dv, dlam, ws) == ar.AR_OK
    assert ar.ar_kernel_launches() == launches and (dlam == 0).all()
