"""Timed cases of what a decoder block does between its matrix products: the
norm and rotation of queries and keys for each head, differential attention
over packed sequences, and the activation whose input is kept in 8 bits for the
backward pass, each in its forward and backward direction.

``own`` selects what ``run`` calls: the library's entry points, or the same
mathematics in elementary torch operations held in 32 bits (angles in 64) and
rounded once at the end.
"""
import math
import random

import torch

own = False

_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_BLOCK = 128  # elements of a row that share a scale


def listed():
    return [
        # Norm and rotation.  A few tokens with GPT-2 small's heads: the call's latency is what counts.
        {"name": "qk fwd 3t 12:12x64 bf16", "op": "qk", "direction": "forward", "tokens": 3, "heads": 12,
         "kv_heads": 12, "dim": 64, "rotary": 64, "interleaved": False, "first": 700, "dtype": "bf16", "params": "bf16"},
        # A batch of a wide model with grouped heads, deep inside a long context.
        {"name": "qk fwd 16384t 32:8x128 bf16", "op": "qk", "direction": "forward", "tokens": 16384, "heads": 32,
         "kv_heads": 8, "dim": 128, "rotary": 128, "interleaved": False, "first": 500000, "dtype": "bf16",
         "params": "f32"},
        # GPT-2 small's heads in f32, half of each head rotated, neighbours paired.
        {"name": "qk bwd 8191t 12:12x64 f32", "op": "qk", "direction": "backward", "tokens": 8191, "heads": 12,
         "kv_heads": 12, "dim": 64, "rotary": 32, "interleaved": True, "first": 0, "dtype": "f32", "params": "f32"},
        # The gradient of the wide model's batch.
        {"name": "qk bwd 16384t 32:8x128 bf16", "op": "qk", "direction": "backward", "tokens": 16384, "heads": 32,
         "kv_heads": 8, "dim": 128, "rotary": 128, "interleaved": False, "first": 0, "dtype": "bf16", "params": "f32"},
        # Differential attention.  A few short sequences, GPT-2 small's width as six heads of two maps: latency.
        {"name": "diff fwd 61t/3 6:6x64 bf16", "op": "diff", "direction": "forward", "tokens": 61, "seqs": 3,
         "heads": 6, "kv_heads": 6, "dim": 64, "vdim": 128, "dtype": "bf16"},
        # One whole long prompt, grouped heads.
        {"name": "diff fwd 8192t/1 16:4x64 bf16", "op": "diff", "direction": "forward", "tokens": 8192, "seqs": 1,
         "heads": 16, "kv_heads": 4, "dim": 64, "vdim": 128, "dtype": "bf16"},
        # GPT-2 small's width over a batch of packed documents of different lengths.
        {"name": "diff bwd 8191t/13 6:6x64 f16", "op": "diff", "direction": "backward", "tokens": 8191, "seqs": 13,
         "heads": 6, "kv_heads": 6, "dim": 64, "vdim": 128, "dtype": "f16"},
        # The gradient of a long packed batch, grouped heads.
        {"name": "diff bwd 8192t/3 16:4x64 bf16", "op": "diff", "direction": "backward", "tokens": 8192, "seqs": 3,
         "heads": 16, "kv_heads": 4, "dim": 64, "vdim": 128, "dtype": "bf16"},
        # The activation.  A few tokens of a hidden layer, forward and backward: latency.
        {"name": "act8 step 5x4096 bf16", "op": "act8", "direction": "step", "rows": 5, "cols": 4096, "pad": 0,
         "kind": "gelu_tanh", "dtype": "bf16"},
        # A residual stream kept for a layer that is computed again: packed and unpacked, in f32.
        {"name": "act8 keep 16384x2048 f32", "op": "act8", "direction": "step", "rows": 16384, "cols": 2048, "pad": 0,
         "kind": "identity", "dtype": "f32"},
        # The backward pass at an odd width, rows inside a wider buffer, with the exact gelu.
        {"name": "act8 bwd 4095x5003 f16", "op": "act8", "direction": "backward", "rows": 4095, "cols": 5003, "pad": 6,
         "kind": "gelu", "dtype": "f16"},
        # The hidden layer of a wide model's batch, forward and backward.
        {"name": "act8 step 16384x10240 bf16", "op": "act8", "direction": "step", "rows": 16384, "cols": 10240,
         "pad": 0, "kind": "gelu_tanh", "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("qk", "diff", "act8"))
    if op == "qk":
        heads, kv = rng.choice(((12, 12), (8, 2), (32, 8), (16, 1), (6, 3), (25, 25)))
        dim = rng.choice((32, 64, 64, 80, 96, 128, 128, 256))
        dtype = rng.choice(("f32", "bf16", "f16"))
        most = min(16384, 167772160 // ((heads + kv) * dim * _SIZE[dtype]))
        return {"op": op, "direction": rng.choice(("forward", "backward")), "tokens": _log(rng, 1, most),
                "heads": heads, "kv_heads": kv, "dim": dim, "rotary": rng.choice((dim, dim, dim // 2)),
                "interleaved": rng.random() < 0.3, "first": rng.choice((0, _log(rng, 1, 1000000))), "dtype": dtype,
                "params": rng.choice(("f32", dtype))}
    if op == "diff":
        heads, kv = rng.choice(((6, 6), (8, 2), (16, 4), (12, 1), (4, 2), (13, 13)))
        dim, vdim = rng.choice(((32, 64), (64, 128), (64, 128), (64, 64), (48, 96), (40, 80)))
        tokens = _log(rng, 8, 8192)
        return {"op": op, "direction": rng.choice(("forward", "backward")), "tokens": tokens,
                "seqs": min(tokens, _log(rng, 1, 48)), "heads": heads, "kv_heads": kv, "dim": dim, "vdim": vdim,
                "dtype": rng.choice(("bf16", "f16"))}
    cols = _log(rng, 64, 20480)
    if rng.random() < 0.5:
        cols = max(8, cols // 8 * 8)  # half of them of the widths that models have
    dtype = rng.choice(("f32", "bf16", "f16"))
    rows = _log(rng, 1, min(32768, 335544320 // (cols * _SIZE[dtype])))
    kind = rng.choice(("gelu_tanh", "gelu_tanh", "gelu", "identity"))
    return {"op": op, "direction": "step" if kind == "identity" else rng.choice(("step", "backward")), "rows": rows,
            "cols": cols, "pad": rng.choice((0, 0, 8, 5)), "kind": kind, "dtype": dtype}


def _lengths(case):
    """The lengths of the packed sequences: they belong to the case, since the
    work depends on them.  Spread over more than a factor of ten; one of ten or
    more sequences is empty, as a batch's padding entry is."""
    n, total = case["seqs"], case["tokens"]
    rng = random.Random(1000003 * total + n)
    if n == 1:
        return [total]
    share = [math.exp(rng.uniform(0.0, 2.5)) for _ in range(n)]
    if n >= 10:
        share[n // 2] = 0.0
    out = [int(total * s / sum(share)) for s in share]
    out[max(range(n), key=lambda i: out[i])] += total - sum(out)
    return out


def work(case):
    b = _SIZE[case["dtype"]]
    forward = case["direction"] == "forward"
    if case["op"] == "qk":
        d, t = case["dim"], case["tokens"]
        n, p = t * (case["heads"] + case["kv_heads"]) * d, _SIZE[case["params"]]
        # a square, a product with rstd, with the weight, and a rotation for each element; twice that and the
        # weight's sums backward
        if forward:
            return {"bytes": 2 * n * b + 2 * d * p + 4 * t, "flops": 7 * n}
        return {"bytes": 3 * n * b + 4 * d * p + 4 * t, "flops": 16 * n}
    if case["op"] == "act8":
        n, s = case["rows"] * case["cols"], case["rows"] * -(-case["cols"] // _BLOCK) * 4
        keep, use = n * b + n + s, n + s  # input read, checkpoint written; checkpoint read
        if case["kind"] == "identity":
            return {"bytes": keep + use + n * b, "flops": 5 * n}
        if case["direction"] == "step":
            return {"bytes": keep + n * b + use + 3 * n * b, "flops": 40 * n}
        return {"bytes": use + 3 * n * b, "flops": 25 * n}
    pairs = sum(n * (n + 1) // 2 for n in _lengths(case))
    t, h, kv, d, e = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["vdim"]
    ins = t * (2 * h * d + 2 * kv * d + kv * e) * b
    if forward:  # both maps' scores, and both maps' products with v, which are both asked for
        return {"bytes": ins + 2 * t * h * e * b + 8 * h * t, "flops": (4 * d + 4 * e) * h * pairs}
    # both maps' scores, dq and dk; dout v^T and dv once
    return {"bytes": 2 * ins + 3 * t * h * e * b + 8 * h * t, "flops": (12 * d + 4 * e) * h * pairs}


# ---- inputs -------------------------------------------------------------------------


def _wide(rows, cols, pad, dtype):
    """A [rows, cols] view of a buffer whose rows are pad elements longer."""
    return torch.empty(rows, cols + pad, device="cuda", dtype=dtype)[:, :cols]


def _prepare_qk(case, g):
    dt, pt = _DTYPE[case["dtype"]], _DTYPE[case["params"]]
    t, h, kv, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]

    def projection():
        # q, k and v are views of one projection's output, as a transformer block has them
        return (torch.randn(t, h + 2 * kv, d, device="cuda", generator=g) *
                (0.5 + 2 * torch.rand(1, h + 2 * kv, 1, device="cuda", generator=g))).to(dt)

    qkv = projection()
    # documents of some hundred tokens one after another, each counted from its own first position
    positions = torch.arange(t, device="cuda") % 777 + case["first"]
    s = {"op": "qk", "direction": case["direction"], "q": qkv[:, :h], "k": qkv[:, h:h + kv], "eps": 1e-6,
         "positions": positions.to(torch.int32), "rotary": case["rotary"], "base": 10000.0,
         "interleaved": case["interleaved"]}
    for n in ("q", "k"):
        s[n + "_weight"] = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(pt)
    if case["direction"] == "forward":
        s.update(q_out=torch.empty(t, h, d, device="cuda", dtype=dt), k_out=torch.empty(t, kv, d, device="cuda", dtype=dt))
    else:
        up, grads = projection(), torch.empty_like(qkv)
        s.update(dq_out=up[:, :h].contiguous(), dk_out=up[:, h:h + kv].contiguous(), dq=grads[:, :h],
                 dk=grads[:, h:h + kv], dq_weight=torch.empty(d, device="cuda", dtype=pt),
                 dk_weight=torch.empty(d, device="cuda", dtype=pt), workspace=None)
    return s


def _prepare_diff(case, g):
    dt = _DTYPE[case["dtype"]]
    t, h, kv, d, e = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["vdim"]
    # the two maps' queries and keys are views of one projection's output, v has its own
    qk = torch.randn(t, 2 * h + 2 * kv, d, device="cuda", generator=g).to(dt)
    ends = torch.tensor([0] + _lengths(case), dtype=torch.int64).cumsum(0)
    s = {"op": "diff", "direction": case["direction"], "q": qk[:, :2 * h], "k": qk[:, 2 * h:],
         "v": torch.randn(t, kv, e, device="cuda", generator=g).to(dt),
         "lam": 0.2 + 0.6 * torch.rand(h, device="cuda", generator=g),
         "cu_seqlens": ends.to(torch.int32).cuda(), "scale": d ** -0.5}
    if case["direction"] == "forward":
        s.update(out=torch.empty(t, h, e, device="cuda", dtype=dt), second=torch.empty(t, h, e, device="cuda", dtype=dt),
                 lse=torch.empty(2 * h, t, device="cuda"))
    else:
        f = _diff_forward(s)
        grads = torch.empty_like(qk)
        s.update(f, dout=torch.randn(t, h, e, device="cuda", generator=g).to(dt), dq=grads[:, :2 * h],
                 dk=grads[:, 2 * h:], dv=torch.empty_like(s["v"]), dlam=torch.empty(h, device="cuda"), workspace=None)
    return s


def _prepare_act8(case, g):
    dt = _DTYPE[case["dtype"]]
    rows, cols, pad = case["rows"], case["cols"], case["pad"]
    x = _wide(rows, cols, pad, dt)
    # what a hidden layer holds before its activation: wider in some columns than in others
    x.copy_(torch.randn(rows, cols, device="cuda", generator=g) *
            torch.exp(0.7 * torch.randn(cols, device="cuda", generator=g)))
    blocks = -(-cols // _BLOCK)
    s = {"op": "act8", "direction": case["direction"], "kind": case["kind"], "rows": rows, "cols": cols, "dtype": dt,
         "again": _wide(rows, cols, pad, dt)}
    if case["kind"] != "identity":
        s.update(dy=_wide(rows, cols, pad, dt), dx=_wide(rows, cols, pad, dt))
        s["dy"].copy_(torch.randn(rows, cols, device="cuda", generator=g))
    if case["direction"] == "backward":
        s["codes"], s["scales"] = _keep(x)
    else:
        s.update(x=x, codes=torch.empty(rows, blocks * _BLOCK, device="cuda", dtype=torch.int8),
                 scales=torch.empty(rows, blocks, device="cuda"))
        if case["kind"] != "identity":
            s["y"] = _wide(rows, cols, pad, dt)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return {"qk": _prepare_qk, "diff": _prepare_diff, "act8": _prepare_act8}[case["op"]](case, g)


# ---- plain forms --------------------------------------------------------------------


def _rotation(s):
    """cos and sin [tokens, 1, rotary / 2] of each pair's angle, which is made in 64 bits."""
    i = torch.arange(s["rotary"] // 2, device="cuda", dtype=torch.float64)
    angle = s["positions"].double()[:, None, None] * s["base"] ** (-2 * i / s["rotary"])
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotate(s, x, cos, sin):
    """The first `rotary` elements of each head as pairs, each turned by its angle."""
    r = s["rotary"]
    out = x.clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if s["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out


def _qk_forward(s):
    cos, sin = _rotation(s)
    r = {}
    for n in ("q", "k"):
        x = s[n].float()
        y = x * (x.square().mean(2, keepdim=True) + s["eps"]).rsqrt() * s[n + "_weight"].float()
        r[n + "_out"] = _rotate(s, y, cos, sin).to(s[n].dtype)
    return r


def _qk_backward(s):
    cos, sin = _rotation(s)
    r = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s[n + "_weight"]
        rstd = (x.square().mean(2, keepdim=True) + s["eps"]).rsqrt()
        g = _rotate(s, s["d" + n + "_out"].float(), cos, -sin)
        xh = x * rstd
        r["d" + n + "_weight"] = (g * xh).sum((0, 1)).to(w.dtype)
        g = g * w.float()
        r["d" + n] = (rstd * (g - xh * (g * xh).mean(2, keepdim=True))).to(s[n].dtype)
    return r


def _diff_scores(s):
    """q and k as [heads, 2, tokens, dim], v as [heads, tokens, vdim], in 32 bits and repeated for their group of
    heads, and the masked scores of both maps."""
    t = s["q"].shape[0]
    h, kv = s["lam"].shape[0], s["v"].shape[1]
    q = s["q"].float().unflatten(1, (h, 2)).permute(1, 2, 0, 3)
    k = s["k"].float().unflatten(1, (kv, 2)).permute(1, 2, 0, 3).repeat_interleave(h // kv, 0)
    v = s["v"].float().transpose(0, 1).repeat_interleave(h // kv, 0)
    at = torch.arange(t, device="cuda")
    seq = torch.searchsorted(s["cu_seqlens"][1:].long(), at, right=True)
    seen = (seq[:, None] == seq[None, :]) & (at[:, None] >= at[None, :])
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    return q, k, v, scores.masked_fill_(~seen, float("-inf"))


def _diff_forward(s):
    q, k, v, scores = _diff_scores(s)
    top = scores.amax(3, keepdim=True)
    e = scores.sub_(top).exp_()
    total = e.sum(3, keepdim=True)
    maps = torch.matmul(e, v[:, None]) / total
    out = maps[:, 0] - s["lam"][:, None, None] * maps[:, 1]
    dt = s["q"].dtype
    return {"out": out.transpose(0, 1).to(dt).contiguous(), "second": maps[:, 1].transpose(0, 1).to(dt).contiguous(),
            "lse": (top + torch.log(total))[..., 0].flatten(0, 1)}


def _diff_backward(s):
    q, k, v, scores = _diff_scores(s)
    h, _, t, d = q.shape
    kv, e = s["v"].shape[1:]
    lam = s["lam"][:, None, None]
    p = scores.sub_(s["lse"].view(h, 2, t, 1)).exp_()
    do, out, second = (s[n].float().transpose(0, 1) for n in ("dout", "out", "second"))
    delta2 = (do * second).sum(2, keepdim=True)
    delta1 = (do * out).sum(2, keepdim=True) + lam * delta2
    dv = torch.matmul((p[:, 0] - lam * p[:, 1]).transpose(1, 2), do).view(kv, h // kv, t, e).sum(1)
    dp = torch.matmul(do, v.transpose(1, 2))
    p[:, 0] *= (dp - delta1) * s["scale"]
    p[:, 1] *= (dp - delta2) * (-s["scale"] * lam)
    dq = torch.matmul(p, k)
    dk = torch.matmul(p.transpose(2, 3), q).view(kv, h // kv, 2, t, d).sum(1)
    dt = s["q"].dtype
    return {"dq": dq.flatten(0, 1).transpose(0, 1).to(dt), "dk": dk.flatten(0, 1).transpose(0, 1).to(dt),
            "dv": dv.transpose(0, 1).to(dt), "dlam": -delta2[..., 0].sum(1)}


def _keep(x):
    """8-bit codes of a matrix, each row filled up with zeros to whole blocks, and the blocks' scales: a code is
    the nearest whole number to x (127 / the block's largest), in 32 bits; a block of less than 2^-120 is zero."""
    rows, cols = x.shape
    blocks = -(-cols // _BLOCK)
    f = torch.zeros(rows, blocks * _BLOCK, device="cuda")
    f[:, :cols] = x
    f = f.view(rows, blocks, _BLOCK)
    top = f.abs().amax(2, keepdim=True)
    some = top >= 2.0 ** -120
    most = torch.full_like(top, 127.0)  # two tensors are divided; a number would be a product with a reciprocal
    codes = torch.where(some, torch.round(f * (most / top)), 0.0)
    return codes.to(torch.int8).view(rows, -1), torch.where(some, top / most, 0.0)[..., 0]


def _kept(s, codes, scales):
    """The values that codes and scales stand for."""
    f = codes.float().view(s["rows"], -1, _BLOCK) * scales[..., None]
    return f.view(s["rows"], -1)[:, :s["cols"]]


def _act(kind, x):
    """The activation and its derivative at x."""
    if kind == "gelu":
        phi = 0.5 * (1 + torch.erf(x * 0.5 ** 0.5))
        return x * phi, phi + x * torch.exp(-0.5 * x * x) * (2 * math.pi) ** -0.5
    c = (2 / math.pi) ** 0.5
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 0.134145 * x * x)


def _act8(s):
    r, dt = {}, s["dtype"]
    codes, scales = _keep(s["x"]) if s["direction"] == "step" else (s["codes"], s["scales"])
    kept = _kept(s, codes, scales)
    if s["kind"] == "identity":
        return {"again": kept.to(dt)}
    if s["direction"] == "step":
        r["y"] = _act(s["kind"], s["x"].float())[0].to(dt)
    again, slope = _act(s["kind"], kept)
    r.update(dx=(s["dy"].float() * slope).to(dt), again=again.to(dt))
    return r


_PLAIN = {("qk", "forward"): _qk_forward, ("qk", "backward"): _qk_backward, ("diff", "forward"): _diff_forward,
          ("diff", "backward"): _diff_backward, ("act8", "step"): _act8, ("act8", "backward"): _act8}


# ---- the library's calls -------------------------------------------------------------


def _own(s):
    from allreduce_gradient_reduction_gb300 import binding as ar
    op, direction = s["op"], s["direction"]
    if op == "qk":
        how = {"rotary_dim": s["rotary"], "base": s["base"], "interleaved": s["interleaved"], "eps": s["eps"]}
        if direction == "forward":
            ar.check(ar.ar_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["q_out"],
                                        s["k_out"], **how))
            return {n: s[n] for n in ("q_out", "k_out")}
        if s["workspace"] is None:
            t, h, d = s["q"].shape
            s["workspace"] = torch.empty(ar.ar_qk_norm_rope_workspace_bytes(t, h, s["k"].shape[1], d), device="cuda",
                                         dtype=torch.uint8)
        ar.check(ar.ar_qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_weight"], s["k_weight"],
                                             s["positions"], s["dq"], s["dk"], s["dq_weight"], s["dk_weight"],
                                             s["workspace"], **how))
        return {n: s[n] for n in ("dq", "dk", "dq_weight", "dk_weight")}
    if op == "diff":
        if direction == "forward":
            ar.check(ar.ar_diff_attention(s["q"], s["k"], s["v"], s["lam"], s["cu_seqlens"], s["out"], s["second"],
                                          s["lse"], scale=s["scale"]))
            return {n: s[n] for n in ("out", "second", "lse")}
        if s["workspace"] is None:
            t, h, e = s["out"].shape
            s["workspace"] = torch.empty(ar.ar_diff_attention_workspace_bytes(t, h, s["v"].shape[1], s["q"].shape[2], e),
                                         device="cuda", dtype=torch.uint8)
        ar.check(ar.ar_diff_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["lam"], s["out"], s["second"],
                                               s["lse"], s["cu_seqlens"], s["dq"], s["dk"], s["dv"], s["dlam"],
                                               s["workspace"], scale=s["scale"]))
        return {n: s[n] for n in ("dq", "dk", "dv", "dlam")}
    r = {}
    if direction == "step":
        ar.check(ar.ar_activation8(s["x"], s.get("y"), s["codes"], s["scales"], kind=s["kind"]))
        if "y" in s:
            r["y"] = s["y"]
    ar.check(ar.ar_activation8_backward(s["codes"], s["scales"], s.get("dy"), s.get("dx"), s["again"], kind=s["kind"]))
    if "dx" in s:
        r["dx"] = s["dx"]
    r["again"] = s["again"]
    return r


def run(state):
    return _own(state) if own else _PLAIN[state["op"], state["direction"]](state)


# ---- the definitions in 64 bits -------------------------------------------------------


def _exact_turn(case, positions):
    """One complex factor for each token and pair."""
    half = case["rotary"] // 2
    freq = torch.tensor([10000.0 ** (-i / half) for i in range(half)], device="cuda", dtype=torch.float64)
    angle = positions.double()[:, None] * freq
    return torch.polar(torch.ones_like(angle), angle)[:, None, :]


def _exact_turned(case, x, turn):
    r, half = case["rotary"], case["rotary"] // 2
    pairs = x[..., :r].unflatten(2, (half, 2)) if case["interleaved"] else x[..., :r].unflatten(2, (2, half)).transpose(2, 3)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.flatten(2) if case["interleaved"] else z.transpose(2, 3).flatten(2)
    return torch.cat((z, x[..., r:]), 2)


def _exact_qk(case, s):
    turn = _exact_turn(case, s["positions"])
    r = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s[n + "_weight"].double()
        norm = torch.sqrt((x * x).mean(2, keepdim=True) + s["eps"])
        if case["direction"] == "forward":
            r[n + "_out"] = _exact_turned(case, x / norm * w, turn)
            continue
        g = _exact_turned(case, s["d" + n + "_out"].double(), turn.conj())
        r["d" + n + "_weight"] = torch.einsum("thd,thd->d", g, x / norm)
        g *= w
        r["d" + n] = g / norm - x * torch.einsum("thd,thd->th", g, x)[..., None] / (case["dim"] * norm ** 3)
    return r


def _exact_diff(case, s):
    t, h, kv, d, e = (case[n] for n in ("tokens", "heads", "kv_heads", "dim", "vdim"))
    big = {"device": "cuda", "dtype": torch.float64}
    forward = case["direction"] == "forward"
    if forward:
        r = {"out": torch.zeros(t, h, e, **big), "second": torch.zeros(t, h, e, **big), "lse": torch.zeros(2 * h, t, **big)}
    else:
        r = {"dq": torch.zeros(t, 2 * h, d, **big), "dk": torch.zeros(t, 2 * kv, d, **big),
             "dv": torch.zeros(t, kv, e, **big), "dlam": torch.zeros(h, **big)}
    start = 0
    for n in _lengths(case):
        at = slice(start, start + n)
        start += n
        mask = torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1)
        for j in range(h if n else 0):
            i, lam = j // (h // kv), s["lam"][j].double()
            v = s["v"][at, i].double()
            p, qs, ks = [], [], []
            for m in (0, 1):
                q, k = s["q"][at, 2 * j + m].double(), s["k"][at, 2 * i + m].double()
                a = (q @ k.T * s["scale"]).masked_fill(mask, -math.inf)
                if forward:
                    r["lse"][2 * j + m, at] = torch.logsumexp(a, 1)
                    p.append(torch.softmax(a, 1))
                else:
                    p.append(torch.exp(a - s["lse"][2 * j + m, at].double()[:, None]))
                qs.append(q)
                ks.append(k)
            if forward:
                r["out"][at, j] = (p[0] - lam * p[1]) @ v
                r["second"][at, j] = p[1] @ v
                continue
            do, second = s["dout"][at, j].double(), s["second"][at, j].double()
            first = s["out"][at, j].double() + lam * second
            r["dv"][at, i] += (p[0] - lam * p[1]).T @ do
            r["dlam"][j] -= (do * second).sum()
            dp = do @ v.T
            for m, o, by in ((0, first, 1.0), (1, second, -lam)):
                da = p[m] * (dp - (do * o).sum(1)[:, None]) * (s["scale"] * by)
                r["dq"][at, 2 * j + m] = da @ ks[m]
                r["dk"][at, 2 * i + m] += da.T @ qs[m]
    return r


def _exact_act8(case, s):
    rows, cols, kind = case["rows"], case["cols"], case["kind"]

    def normal(x):  # the normal distribution's integral, exact at both ends
        return 0.5 * torch.special.erfc(-x / math.sqrt(2))

    def act(x):
        if kind == "gelu":
            return x * normal(x)
        return x * torch.sigmoid(math.sqrt(8 / math.pi) * (x + 0.044715 * x ** 3))

    def slope(x):
        if kind == "gelu":
            return normal(x) + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        u = math.sqrt(8 / math.pi) * (x + 0.044715 * x ** 3)
        g = torch.sigmoid(u)
        return g + x * g * torch.sigmoid(-u) * math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * x * x)

    parts = []
    step = max(1, 60000000 // cols)
    for a in range(0, rows, step):
        at = slice(a, min(rows, a + step))
        n = at.stop - a
        out = {}
        if case["direction"] == "step":
            # a code is defined by one division and one product of binary32: both are rounded to it here
            x = s["x"][at].double()
            full = torch.nn.functional.pad(x, (0, -cols % _BLOCK)).view(n, -1, _BLOCK)
            top = full.abs().max(2, keepdim=True).values
            by = (127.0 / top.clamp(min=1e-300)).float().double()
            code = torch.round((full * by).float()).double() * (top >= 2.0 ** -120)
            kept = (code * (top / 127.0).float().double()).view(n, -1)[:, :cols]
            if kind != "identity":
                out["y"] = act(x)
        else:
            kept = (s["codes"][at].double().view(n, -1, _BLOCK) * s["scales"][at].double()[..., None]).view(n, -1)[:, :cols]
        if kind == "identity":
            out["again"] = kept
        else:
            out.update(dx=s["dy"][at].double() * slope(kept), again=act(kept))
        parts.append(out)
    return {n: torch.cat([p[n] for p in parts]) for n in parts[0]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"qk": _exact_qk, "diff": _exact_diff, "act8": _exact_act8}[case["op"]](case, s)
