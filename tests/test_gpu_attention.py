"""ar_attention and ar_attention_backward against the formulas in 64 bits.

Tolerances.  u is the tensors' unit roundoff: half the spacing above 1, 2^-8
bf16 (8 significant bits), 2^-11 f16.  A result is rounded once (u of itself),
and so is every probability (or ds) before the product that sums it: u of the
sum of the terms' magnitudes.  Scores, and the products dout.v and dout.out, are binary32 sums
of exact products of at most 128 terms: off by at most 2^-17 of the sum of the
terms' magnitudes, which enters a probability as a relative error; the
exponential adds a few units of its exponent, which stays below 2^-13 here.
Probabilities below the smallest normal number of f16 are off by 2^-25 of the
row's largest, which is at least one; results there are off by the same
2^-25 (half of f16's spacing).
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


def packed(lengths, before=0):
    return torch.tensor(np.cumsum([before] + list(lengths)), dtype=torch.int32, device="cuda")


def make(tokens, heads, kv, dim, dtype, seed, n=1, amplitude=1.0):
    """n tensors of each of [tokens, heads, dim] and [tokens, kv, dim]"""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    shape = [(heads, n), (kv, 2)]
    return [(torch.randn(tokens, h, dim, device="cuda", generator=g) * amplitude).to(DT[dtype])
            for h, k in shape for _ in range(k)]


def sequences(cu):
    c = cu.tolist()
    return [(a, b) for a, b in zip(c, c[1:]) if b > a]


def reference(q, k, v, cu, scale, dout=None, out=None, lse=None):
    """Results and their tolerances' parts.  Forward: (out, lse, sum of p|v|,
    error of a score, |v| sums); backward: dq, dk, dv with theirs."""
    t, h, d = q.shape
    group = h // k.shape[1]
    r = {}

    def put(name, shape, at, value):
        r.setdefault(name, np.zeros(shape))[at] += value

    for a, b in sequences(cu):
        n = b - a
        mask = np.triu(np.ones((n, n), bool), 1)
        for j in range(h):
            Q, K, V = f64(q[a:b, j]), f64(k[a:b, j // group]), f64(v[a:b, j // group])
            s = Q @ K.T * scale
            s[mask] = -np.inf
            size = (np.abs(Q) @ np.abs(K).T * scale * ~mask).max(1)
            if dout is None:
                top = s.max(1, keepdims=True)
                e = np.exp(s - top)
                p = e / e.sum(1, keepdims=True)
                at = (slice(a, b), j)
                put("out", (t, h, d), at, p @ V)
                put("lse", (t, h), at, (top + np.log(e.sum(1, keepdims=True)))[:, 0])
                put("weight", (t, h, d), at, p @ np.abs(V))
                put("all", (t, h, d), at, ~mask @ np.abs(V))
                put("size", (t, h), at, size)
                continue
            DO, O = f64(dout[a:b, j]), f64(out[a:b, j])
            p = np.exp(s - f64(lse[j, a:b])[:, None])
            dp = DO @ V.T
            ds = p * (dp - (DO * O).sum(1, keepdims=True))
            off = np.abs(ds) * (EXP + SCORE * size[:, None]) + p * SCORE * (
                np.abs(DO) @ np.abs(V).T + (np.abs(DO) * np.abs(O)).sum(1, keepdims=True))
            at, kat = (slice(a, b), j), (slice(a, b), j // group)
            put("dq", (t, h, d), at, scale * ds @ K)
            put("dk", k.shape, kat, scale * ds.T @ Q)
            put("dv", k.shape, kat, p.T @ DO)
            put("dq_terms", (t, h, d), at, scale * np.abs(ds) @ np.abs(K))
            put("dk_terms", k.shape, kat, scale * np.abs(ds).T @ np.abs(Q))
            put("dv_terms", k.shape, kat, p.T @ np.abs(DO))
            put("dq_off", (t, h, d), at, scale * off @ np.abs(K))
            put("dk_off", k.shape, kat, scale * off.T @ np.abs(Q))
            put("dv_off", k.shape, kat, (p * (EXP + SCORE * size[:, None])).T @ np.abs(DO))
            put("dq_all", (t, h, d), at, scale * ~mask @ np.abs(K))
            put("dk_all", k.shape, kat, scale * (~mask).T @ np.abs(Q))
            put("dv_all", k.shape, kat, (~mask).T @ np.abs(DO))
    return r


def within(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3])


def covered(cu, tokens):
    c = np.zeros(tokens, bool)
    for a, b in sequences(cu):
        c[a:b] = True
    return c


def check(ar, q, k, v, cu, dtype, dout=None, scale=None, out=None, grads=None):
    t, h, d = q.shape
    kv = k.shape[1]
    s = d ** -0.5 if scale is None else scale
    out = torch.full((t, h, d), 7.0, dtype=DT[dtype], device="cuda") if out is None else out
    lse = torch.full((h, t), 7.0, device="cuda")
    ar.check(ar.ar_attention(q, k, v, cu, out, lse, scale=scale), "ar_attention")
    assert ar.ar_device_status() == (0, 0)
    r = reference(q, k, v, cu, s)
    on = covered(cu, t)
    got = f64(out)
    if on.any():
        rel = EXP + SCORE * r["size"][..., None]
        within(got[on], r["out"][on], (U[dtype] * np.abs(r["out"]) + (U[dtype] + rel) * r["weight"]
                                      + LOST[dtype] * (1 + r["all"]))[on], "out")
        within(f64(lse).T[on], r["lse"][on], (SCORE * r["size"] + 2.0 ** -18 * (1 + np.abs(r["lse"])))[on], "lse")
    assert (got[~on] == 7).all() and (f64(lse).T[~on] == 7).all()  # tokens of no sequence
    if dout is None:
        return out, lse
    if grads is None:
        grads = [torch.full_like(x, 7.0, memory_format=torch.contiguous_format) for x in (q, k, v)]
    ws = torch.full((ar.ar_attention_workspace_bytes(t, h, kv, d),), 0xFF, dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_attention_backward(dout, q, k, v, out, lse, cu, *grads, ws, scale=scale), "ar_attention_backward")
    assert ar.ar_device_status() == (0, 0)
    if on.any():
        r = reference(q, k, v, cu, s, dout, out, lse)
    for x, name in zip(grads, ("dq", "dk", "dv")):
        if on.any():
            tol = U[dtype] * np.abs(r[name]) + U[dtype] * r[name + "_terms"] + 2 * r[name + "_off"] \
                + LOST[dtype] * (1 + r[name + "_all"])
            within(f64(x)[on], r[name][on], tol[on], name)
        assert (f64(x)[~on] == 7).all()
    return out, lse, grads


LENGTHS = [[1], [2], [127], [128], [129], [255], [256], [257], [300, 1, 0, 77, 128], [1, 1, 1], [513], [64, 640]]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_lengths(ar, lengths, dim, dtype):
    q, k, v = make(sum(lengths), 2, 1, dim, dtype, 1)
    dout = make(sum(lengths), 2, 1, dim, dtype, 2)[0]
    check(ar, q, k, v, packed(lengths), dtype, dout)


@pytest.mark.parametrize("dim", [8, 16, 24, 32, 40, 72, 80, 96, 104, 120])
def test_head_sizes(ar, dim):
    q, k, v = make(200, 3, 3, dim, "bf16", 3)
    dout = make(200, 3, 3, dim, "bf16", 4)[0]
    check(ar, q, k, v, packed([150, 50]), "bf16", dout)


@pytest.mark.parametrize("heads,kv", [(1, 1), (12, 12), (8, 2), (6, 1), (32, 8)])
@pytest.mark.parametrize("dim", [64, 128])
def test_shared_heads(ar, heads, kv, dim):
    q, k, v = make(290, heads, kv, dim, "f16", 5)
    dout = make(290, heads, kv, dim, "f16", 6)[0]
    check(ar, q, k, v, packed([131, 159]), "f16", dout)


def test_many_sequences(ar):
    """More sequences than a warp looks at at once, empty ones among them."""
    g = np.random.Generator(np.random.PCG64(7))
    lengths = [int(x) for x in g.integers(0, 40, 150)]
    lengths[70] = 400
    t = sum(lengths)
    q, k, v = make(t, 2, 2, 64, "bf16", 8)
    dout = make(t, 2, 2, 64, "bf16", 9)[0]
    check(ar, q, k, v, packed(lengths), "bf16", dout)


def test_long_sequence(ar):
    q, k, v = make(2111, 2, 1, 128, "bf16", 10)
    dout = make(2111, 2, 1, 128, "bf16", 11)[0]
    check(ar, q, k, v, packed([2111]), "bf16", dout)


@pytest.mark.parametrize("dim", [64, 128])
def test_growing_scores(ar, dim):
    """Keys that grow along the sequence, so that a row's maximum keeps moving
    and the output is rescaled again and again."""
    q, k, v = make(1100, 2, 2, dim, "f16", 12)
    q = q.abs() * 0.5
    k = (k.abs() * 0.25 + torch.arange(1100, device="cuda")[:, None, None] / 250).to(k.dtype)
    dout = make(1100, 2, 2, dim, "f16", 13)[0]
    check(ar, q, k, v, packed([1100]), "f16", dout)


def test_scale(ar):
    q, k, v = make(140, 2, 2, 64, "bf16", 14)
    dout = make(140, 2, 2, 64, "bf16", 15)[0]
    for scale in (0.02, 0.5):
        check(ar, q, k, v, packed([140]), "bf16", dout, scale=scale)


def test_tokens_outside_every_sequence(ar):
    q, k, v = make(500, 2, 1, 64, "bf16", 16)
    dout = make(500, 2, 1, 64, "bf16", 17)[0]
    check(ar, q, k, v, packed([200, 130], before=37), "bf16", dout)
    check(ar, q, k, v, packed([0, 0], before=3), "bf16", dout)


@pytest.mark.parametrize("layout", ["one projection", "heads outside", "padded", "heads in any order"])
def test_layouts(ar, layout):
    t, h, kv, d, dtype = 333, 4, 2, 64, "bf16"
    q0, k0, v0 = make(t, h, kv, d, dtype, 18)
    dout0 = make(t, h, kv, d, dtype, 19)[0]

    def place(parts):
        if layout == "one projection":
            whole = torch.cat(parts, 1).contiguous()
            return list(torch.split(whole, [p.shape[1] for p in parts], 1))
        if layout == "heads outside":
            return [p.transpose(0, 1).contiguous().transpose(0, 1) for p in parts]
        if layout == "padded":
            return [torch.nn.functional.pad(p, (0, 24, 0, 1))[:, :-1, :d] for p in parts]
        return [torch.cat([p, p], 1)[:, ::2] if p.shape[1] == 1 else
                torch.stack([p, torch.zeros_like(p)], 2)[:, :, 0] for p in parts]

    q, k, v = place([q0, k0, v0])
    (dout,), (out,) = place([dout0]), place([torch.full_like(q0, 7.0)])
    grads = place([torch.full_like(x, 7.0) for x in (q0, k0, v0)])
    check(ar, q, k, v, packed([200, 133]), dtype, dout, out=out, grads=grads)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_sequences_do_not_matter(ar, bad, dim):
    """Every tensor of the middle sequence, and of the tokens after the last,
    is not finite: the others' results keep their bits."""
    t, lengths = 700, [130, 250, 190]
    q, k, v = make(t, 2, 1, dim, "bf16", 20)
    dout = make(t, 2, 1, dim, "bf16", 21)[0]
    cu = packed(lengths)
    clean = check(ar, q, k, v, cu, "bf16", dout)
    results = [clean[0], clean[1].t(), *clean[2]]
    q2, k2, v2, do2 = (x.clone() for x in (q, k, v, dout))
    for x in (q2, k2, v2, do2):
        x[130:380] = bad
        x[570:] = bad
    out, lse = torch.empty_like(q), torch.empty(2, t, device="cuda")
    grads = [torch.empty_like(x) for x in (q, k, v)]
    ws = torch.empty(ar.ar_attention_workspace_bytes(t, 2, 1, dim), dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_attention(q2, k2, v2, cu, out, lse), "forward")
    ar.check(ar.ar_attention_backward(do2, q2, k2, v2, out, lse, cu, *grads, ws), "backward")
    for a, b in zip(results, (out, lse.t(), *grads)):
        for at in (slice(0, 130), slice(380, 570)):
            assert torch.equal(a[at], b[at])


def test_later_keys_do_not_matter(ar):
    """Scores of later tokens may be anything; values that are not finite reach
    no token more than 127 before their own."""
    q, k, v = make(400, 2, 1, 64, "bf16", 22)
    cu = packed([400])
    out, lse = check(ar, q, k, v, cu, "bf16")
    k2, v2 = k.clone(), v.clone()
    k2[300:] = float("nan")
    v2[390:] = float("inf")
    got, got_lse = torch.empty_like(out), torch.empty_like(lse)
    ar.check(ar.ar_attention(q, k2, v2, cu, got, got_lse), "forward")
    assert torch.equal(got[:263], out[:263]) and torch.equal(got_lse[:, :300], lse[:, :300])
    assert torch.isnan(got[300:]).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens", [100, 300, 449])
def test_a_key_of_minus_infinity(ar, tokens, dim):
    """A key whose scores are all -inf has no weight: it and its value get zero
    gradients, others finite ones, also where the last tile of queries is cut."""
    q, k, v = make(tokens, 2, 1, dim, "bf16", 40)
    dout = make(tokens, 2, 1, dim, "bf16", 41)[0]
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    k[5, :, 0] = -float("inf")
    cu = packed([tokens])
    out, lse = torch.empty_like(q), torch.empty(2, tokens, device="cuda")
    dq, dk, dv = (torch.full_like(x, 7.0) for x in (q, k, v))
    ws = torch.empty(ar.ar_attention_workspace_bytes(tokens, 2, 1, dim), dtype=torch.uint8, device="cuda")
    ar.check(ar.ar_attention(q, k, v, cu, out, lse), "forward")
    ar.check(ar.ar_attention_backward(dout, q, k, v, out, lse, cu, dq, dk, dv, ws), "backward")
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert (dk[5] == 0).all() and (dv[5] == 0).all()
    assert torch.isfinite(dk).all() and torch.isfinite(dv).all() and torch.isfinite(dq[:, :, 1:]).all()


def test_first_token_sees_itself_alone(ar):
    q, k, v = make(50, 2, 2, 64, "f16", 23)
    cu = packed([1, 30, 19])
    out, lse = check(ar, q, k, v, cu, "f16")
    for first in (0, 1, 31):
        assert torch.equal(out[first], v[first])


def test_gradient_agrees_with_differences(ar):
    """dq, dk and dv against central differences of the formula's sum(out *
    dout) in 64 bits: at a step of 1e-4 their own error is below 1e-6 of the
    terms; the gradients' is at most u twice, for each of their terms."""
    lengths, scale, h = [5, 9], 0.3, 1e-4
    q, k, v = make(14, 4, 2, 16, "f16", 24)
    dout = make(14, 4, 2, 16, "f16", 25)[0]
    cu = packed(lengths)
    _, _, grads = check(ar, q, k, v, cu, "f16", dout, scale=scale)

    def total(*x):
        return (reference(*x, cu, scale)["out"] * f64(dout)).sum()

    g = torch.Generator(device="cuda")
    g.manual_seed(26)
    base = [x.double() for x in (q, k, v)]
    for _ in range(6):
        d = [torch.randn(x.shape, device="cuda", generator=g, dtype=torch.float64) for x in base]
        up = total(*(x + h * e for x, e in zip(base, d)))
        down = total(*(x - h * e for x, e in zip(base, d)))
        got = sum((x.double() * e).sum().item() for x, e in zip(grads, d))
        size = sum((x.double() * e).abs().sum().item() for x, e in zip(grads, d))
        assert abs((up - down) / (2 * h) - got) <= 4 * U["f16"] * size


def test_same_bits_on_another_stream_and_in_a_graph(ar):
    t = 600
    q, k, v = make(t, 4, 2, 64, "bf16", 27)
    dout = make(t, 4, 2, 64, "bf16", 28)[0]
    cu = packed([250, 350])
    out, lse, grads = check(ar, q, k, v, cu, "bf16", dout)
    got = [torch.zeros_like(x) for x in (out, lse, *grads)]
    ws = torch.empty(ar.ar_attention_workspace_bytes(t, 4, 2, 64), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ar.check(ar.ar_attention(q, k, v, cu, got[0], got[1]), "forward")
        ar.check(ar.ar_attention_backward(dout, q, k, v, got[0], got[1], cu, *got[2:], ws), "backward")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for x in got:
            x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, lse, *grads)))


def test_without_lse(ar):
    q, k, v = make(70, 2, 2, 64, "bf16", 29)
    cu = packed([70])
    out, _ = check(ar, q, k, v, cu, "bf16")
    got = torch.empty_like(out)
    ar.check(ar.ar_attention(q, k, v, cu, got), "no lse")
    assert torch.equal(got, out)


def test_lengths_that_are_not_sound_stay_inside_the_tensors(ar):
    """Entries outside [0, tokens] are clamped, a decreasing pair is an empty
    sequence."""
    q, k, v = make(100, 2, 2, 64, "bf16", 30)
    whole, _ = check(ar, q, k, v, packed([100]), "bf16")
    out = torch.zeros_like(q)
    cu = torch.tensor([-5, 1000], dtype=torch.int32, device="cuda")
    ar.check(ar.ar_attention(q, k, v, cu, out), "clamped")
    assert torch.equal(out, whole)
    out.zero_()
    cu = torch.tensor([60, 20], dtype=torch.int32, device="cuda")
    ar.check(ar.ar_attention(q, k, v, cu, out), "decreasing")
    assert (out == 0).all() and ar.ar_device_status() == (0, 0)


def test_refusals(ar):
    q, k, v = make(40, 4, 2, 64, "bf16", 31)
    out, lse, cu = torch.empty_like(q), torch.empty(4, 40, device="cuda"), packed([40])
    bad, unsupported = ar.AR_ERR_INVALID_ARG, ar.AR_ERR_UNSUPPORTED
    launches = ar.ar_kernel_launches()
    assert ar.ar_attention(q.float(), k.float(), v.float(), cu, out.float(), lse) == unsupported
    assert ar.ar_attention(q.int(), k.int(), v.int(), cu, out.int(), lse) == unsupported
    assert ar.ar_attention(q, k.half(), v, cu, out, lse) == bad
    assert ar.ar_attention(q, k[:, :, :32], v, cu, out, lse) == bad
    assert ar.ar_attention(q[:, :3], k, v, cu, out[:, :3], lse[:3]) == bad       # 3 heads over 2
    assert ar.ar_attention(q, k, v, cu.long(), out, lse) == bad
    assert ar.ar_attention(q, k, v, cu.cpu(), out, lse) == bad
    assert ar.ar_attention(q, k, v, cu, out[:39], lse) == bad
    assert ar.ar_attention(q, k, v, cu, out, lse[:3]) == bad
    assert ar.ar_attention(q, k, v, cu, q, lse) == bad                          # not in place
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert ar.ar_attention(q, k, v, cu, out, lse, scale=scale) == bad
    # sizes and strides that are no multiples of eight, starts that are not on 16 bytes, too large heads
    odd = torch.zeros(40, 4, 100, dtype=torch.bfloat16, device="cuda")
    assert ar.ar_attention(odd, odd, odd, cu, torch.empty_like(odd)) == unsupported
    assert ar.ar_attention(odd[:, :, :64], k, v, cu, out, lse) == bad
    wide = torch.zeros(40, 4, 72, dtype=torch.bfloat16, device="cuda")
    assert ar.ar_attention(wide[:, :, 1:65], k, v, cu, out, lse) == bad
    assert ar.ar_attention(wide[:, :, 8:72], k, v, cu, out, lse) == ar.AR_OK
    big = torch.zeros(40, 4, 136, dtype=torch.bfloat16, device="cuda")
    assert ar.ar_attention(big, big, big, cu, torch.empty_like(big)) == unsupported
    assert ar.ar_attention(q[:1].expand(40, 4, 64), k, v, cu, out, lse) == bad
    launches += 1
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(ar.ar_attention_workspace_bytes(40, 4, 2, 64), dtype=torch.uint8, device="cuda")
    args = (out, q, k, v, out, lse, cu)
    assert ar.ar_attention_backward(*args, dq, dk, dv, ws[:-1]) == bad
    assert ar.ar_attention_backward(*args, dq, dk, dk, ws) == bad
    assert ar.ar_attention_backward(*args, q, dk, dv, ws) == bad
    assert ar.ar_attention_backward(out, q, k, v, out, None, cu, dq, dk, dv, ws) == bad
    assert ar.ar_kernel_launches() == launches
    assert ar.ar_attention_workspace_bytes(40, 3, 2, 64) == bad
    # nothing to do
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert ar.ar_attention(none, none[:, :2], none[:, :2], cu, none) == ar.AR_OK
    assert ar.ar_attention(q, k, v, cu[:1], out, lse) == ar.AR_OK
    assert ar.ar_kernel_launches() == launches
