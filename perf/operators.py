"""Timed cases of the training-step operators: layer norm, causal attention
over packed sequences and the distillation loss, each in its forward and
backward direction.

``own`` selects what ``run`` calls: the library's entry points, or the same
mathematics in elementary torch operations held in 32 bits and rounded once
at the end.
"""
import math
import random

import torch

own = False

_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # Layer norm.  A few tokens of GPT-2 small's width: the call's latency is what counts.
        {"name": "ln fwd 4x768 bf16", "op": "ln", "direction": "forward", "rows": 4, "cols": 768, "pad": 0,
         "dtype": "bf16", "params": "bf16"},
        # A batch of 16 sequences of 1024 tokens of a wide model with an odd width, rows inside a wider buffer.
        {"name": "ln fwd 16384x5121 bf16", "op": "ln", "direction": "forward", "rows": 16384, "cols": 5121, "pad": 7,
         "dtype": "bf16", "params": "f32"},
        # GPT-2 small in f32: 8 sequences of 1024 tokens.
        {"name": "ln bwd 8192x768 f32", "op": "ln", "direction": "backward", "rows": 8192, "cols": 768, "pad": 0,
         "dtype": "f32", "params": "f32"},
        # A wide model's batch in bf16, with parameters and their gradients in f32.
        {"name": "ln bwd 32768x4096 bf16", "op": "ln", "direction": "backward", "rows": 32768, "cols": 4096, "pad": 0,
         "dtype": "bf16", "params": "f32"},
        # Distillation.  A handful of tokens over GPT-2's vocabulary: few rows, so one row has to be spread out.
        {"name": "distill step 6x50257 bf16", "op": "distill", "direction": "step", "rows": 6, "vocab": 50257,
         "top": 16, "pad": 0, "dtype": "bf16", "temperature": 2.0},
        # Evaluation of the loss alone in f32.
        {"name": "distill fwd 2048x50257 f32", "op": "distill", "direction": "forward", "rows": 2048, "vocab": 50257,
         "top": 64, "pad": 0, "dtype": "f32", "temperature": 1.0},
        # A training step's loss and gradient in one call: 8 sequences of 1024 tokens.
        {"name": "distill step 8192x50257 bf16", "op": "distill", "direction": "step", "rows": 8192, "vocab": 50257,
         "top": 64, "pad": 0, "dtype": "bf16", "temperature": 2.0},
        # The gradient for an upstream one, over a large vocabulary, rows inside a wider buffer.
        {"name": "distill bwd 1023x128003 f16", "op": "distill", "direction": "backward", "rows": 1023,
         "vocab": 128003, "top": 100, "pad": 5, "dtype": "f16", "temperature": 1.5},
        # Attention.  A few short sequences with GPT-2 small's heads: latency.
        {"name": "attn fwd 61t/3 12x64 bf16", "op": "attn", "direction": "forward", "tokens": 61, "seqs": 3,
         "heads": 12, "kv_heads": 12, "dim": 64, "dtype": "bf16"},
        # One whole long prompt, grouped heads of 128.
        {"name": "attn fwd 8192t/1 32:8x128 bf16", "op": "attn", "direction": "forward", "tokens": 8192, "seqs": 1,
         "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16"},
        # GPT-2 small's heads over a batch of packed documents of different lengths.
        {"name": "attn bwd 8191t/13 12x64 f16", "op": "attn", "direction": "backward", "tokens": 8191, "seqs": 13,
         "heads": 12, "kv_heads": 12, "dim": 64, "dtype": "f16"},
        # The gradient of a long packed batch, grouped heads of 128.
        {"name": "attn bwd 8192t/3 32:8x128 bf16", "op": "attn", "direction": "backward", "tokens": 8192, "seqs": 3,
         "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("ln", "distill", "attn"))
    if op == "ln":
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.5:
            cols = max(8, cols // 8 * 8)  # half of them of the widths that models have
        rows = _log(rng, 1, min(32768, 134217728 // cols))
        dtype = rng.choice(("f32", "bf16", "f16"))
        return {"op": op, "direction": rng.choice(("forward", "backward")), "rows": rows, "cols": cols,
                "pad": rng.choice((0, 0, 8, 5)), "dtype": dtype, "params": rng.choice(("f32", dtype))}
    if op == "distill":
        vocab = _log(rng, 1000, 131072)
        rows = _log(rng, 1, min(8192, 200000000 // vocab))
        return {"op": op, "direction": rng.choice(("forward", "step", "backward")), "rows": rows, "vocab": vocab,
                "top": min(vocab, _log(rng, 1, 128)), "pad": rng.choice((0, 0, 8, 3)),
                "dtype": rng.choice(("f32", "bf16", "f16")), "temperature": rng.choice((1.0, 2.0, 3.5))}
    heads, kv = rng.choice(((12, 12), (8, 2), (32, 8), (16, 1), (6, 3), (25, 25)))
    tokens = _log(rng, 8, 8192)
    return {"op": op, "direction": rng.choice(("forward", "backward")), "tokens": tokens,
            "seqs": min(tokens, _log(rng, 1, 48)), "heads": heads, "kv_heads": kv,
            "dim": rng.choice((32, 64, 64, 80, 96, 128, 128)), "dtype": rng.choice(("bf16", "f16"))}


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
    if case["op"] == "ln":
        n, c, r = case["rows"] * case["cols"], case["cols"], case["rows"]
        p = _SIZE[case["params"]]
        if case["direction"] == "forward":
            return {"bytes": 2 * n * b + 2 * c * p + 8 * r, "flops": 8 * n}
        return {"bytes": 3 * n * b + 3 * c * p + 8 * r, "flops": 14 * n}
    if case["op"] == "distill":
        n, r = case["rows"] * case["vocab"], case["rows"]
        lists = r * case["top"] * 8
        passes = 1 if case["direction"] == "forward" else 2
        return {"bytes": passes * n * b + lists + 12 * r, "flops": (4 if passes == 1 else 7) * n}
    pairs = sum(n * (n + 1) // 2 for n in _lengths(case))
    t, h, kv, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    if case["direction"] == "forward":
        return {"bytes": (2 * h + 2 * kv) * t * d * b + 4 * h * t, "flops": 4 * d * h * pairs}
    return {"bytes": (4 * h + 4 * kv) * t * d * b + 4 * h * t, "flops": 10 * d * h * pairs}


# ---- inputs -------------------------------------------------------------------------


def _wide(rows, cols, pad, dtype):
    """A [rows, cols] view of a buffer whose rows are pad elements longer."""
    return torch.empty(rows, cols + pad, device="cuda", dtype=dtype)[:, :cols]


def _prepare_ln(case, g):
    dt, pt = _DTYPE[case["dtype"]], _DTYPE[case["params"]]
    rows, cols, pad = case["rows"], case["cols"], case["pad"]
    x = _wide(rows, cols, pad, dt)
    # activations with a spread and an offset of their own in each row, as residual streams have
    spread = torch.rand(rows, 1, device="cuda", generator=g) * 2 + 0.5
    offset = torch.randn(rows, 1, device="cuda", generator=g) * 0.5
    x.copy_(torch.randn(rows, cols, device="cuda", generator=g) * spread + offset)
    s = {"op": "ln", "direction": case["direction"], "x": x, "eps": 1e-5,
         "weight": (1 + 0.1 * torch.randn(cols, device="cuda", generator=g)).to(pt),
         "bias": (0.1 * torch.randn(cols, device="cuda", generator=g)).to(pt)}
    if case["direction"] == "forward":
        s.update(y=torch.empty(rows, cols, device="cuda", dtype=dt),
                 mean=torch.empty(rows, device="cuda"), rstd=torch.empty(rows, device="cuda"))
    else:
        f = x.float()
        s["mean"] = f.mean(1)
        s["rstd"] = ((f - s["mean"][:, None]).square().mean(1) + s["eps"]).rsqrt()
        s.update(dy=torch.randn(rows, cols, device="cuda", generator=g).to(dt),
                 dx=torch.empty(rows, cols, device="cuda", dtype=dt),
                 dweight=torch.empty(cols, device="cuda", dtype=pt), dbias=torch.empty(cols, device="cuda", dtype=pt))
    return s


def _prepare_distill(case, g):
    dt = _DTYPE[case["dtype"]]
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    logits = _wide(rows, vocab, case["pad"], dt)
    logits.copy_(torch.randn(rows, vocab, device="cuda", generator=g) * 2)
    # the teacher's list: its own logits at words that it prefers, highest first
    index = torch.randint(vocab, (rows, top), device="cuda", generator=g)
    index = (index[:, :1] + torch.arange(top, device="cuda") * max(1, vocab // top)) % vocab
    value = torch.gather(logits.float(), 1, index) * 0.5 + torch.randn(rows, top, device="cuda", generator=g) * 2 + 3
    value, order = torch.sort(value, dim=1, descending=True)
    index = torch.gather(index, 1, order).to(torch.int32)
    # some lists are shorter, and a row in sixteen (a padding token) has none
    kept = torch.randint(top // 2 + 1, top + 1, (rows, 1), device="cuda", generator=g)
    kept[15::16] = 0
    index[torch.arange(top, device="cuda") >= kept] = -1
    scale = torch.full((rows,), 1.0 / rows, device="cuda")
    s = {"op": "distill", "direction": case["direction"], "logits": logits, "index": index, "value": value,
         "temperature": case["temperature"], "scale": scale}
    if case["direction"] == "backward":
        s["lse"] = torch.logsumexp(logits.float() / case["temperature"], 1)
        s["scale"] = torch.rand(rows, device="cuda", generator=g) + 0.5
    else:
        s.update(loss=torch.empty(rows, device="cuda"), lse=torch.empty(rows, device="cuda"))
    if case["direction"] != "forward":
        s["dlogits"] = _wide(rows, vocab, case["pad"], dt)
    return s


def _prepare_attn(case, g):
    dt = _DTYPE[case["dtype"]]
    t, h, kv, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    # q, k and v are views of one projection's output, as a transformer block has them
    qkv = torch.randn(t, h + 2 * kv, d, device="cuda", generator=g).to(dt)
    ends = torch.tensor([0] + _lengths(case), dtype=torch.int64).cumsum(0)
    s = {"op": "attn", "direction": case["direction"], "q": qkv[:, :h], "k": qkv[:, h:h + kv], "v": qkv[:, h + kv:],
         "cu_seqlens": ends.to(torch.int32).cuda(), "scale": d ** -0.5, "workspace": None}
    if case["direction"] == "forward":
        s.update(out=torch.empty(t, h, d, device="cuda", dtype=dt), lse=torch.empty(h, t, device="cuda"))
    else:
        f = _attn_forward(s)
        grads = torch.empty_like(qkv)
        s.update(out=f["out"], lse=f["lse"], dout=torch.randn(t, h, d, device="cuda", generator=g).to(dt),
                 dq=grads[:, :h], dk=grads[:, h:h + kv], dv=grads[:, h + kv:])
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return {"ln": _prepare_ln, "distill": _prepare_distill, "attn": _prepare_attn}[case["op"]](case, g)


# ---- plain forms --------------------------------------------------------------------


def _ln_forward(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = (d.square().mean(1, keepdim=True) + s["eps"]).rsqrt()
    y = d * rstd * s["weight"].float() + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _ln_backward(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    pt = s["weight"].dtype
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0).to(pt), "dbias": dy.sum(0).to(pt)}


def _distill_teacher(s):
    """The teacher's probabilities over each row's list (0 where it has no entry) and their logarithms."""
    there = s["index"] >= 0
    t = torch.where(there, s["value"] / s["temperature"], float("-inf"))
    top = t.amax(1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    e = torch.exp(t - top)
    total = e.sum(1, keepdim=True)
    some = total > 0
    p = torch.where(some, e / total, 0.0)
    logp = torch.where(p > 0, t - top - torch.log(total), 0.0)
    return p, logp, some, s["index"].clamp_min(0).long()


def _distill_gradient(s, z, lse, p, some, at):
    q = torch.exp(z - lse[:, None])
    grad = q.scatter_add(1, at, -p) * (s["scale"] * s["temperature"])[:, None]
    return torch.where(some & (s["scale"] != 0)[:, None], grad, 0.0).to(s["logits"].dtype)


def _distill_forward(s):
    z = s["logits"].float() / s["temperature"]
    top = z.amax(1, keepdim=True)
    lse = (top + torch.log(torch.exp(z - top).sum(1, keepdim=True)))[:, 0]
    p, logp, some, at = _distill_teacher(s)
    logq = torch.gather(z, 1, at) - lse[:, None]
    loss = torch.where(p > 0, p * (logp - logq), 0.0).sum(1) * s["temperature"] ** 2
    r = {"loss": loss, "lse": lse}
    if s["direction"] == "step":
        r["dlogits"] = _distill_gradient(s, z, lse, p, some, at)
    return r


def _distill_backward(s):
    p, _, some, at = _distill_teacher(s)
    return {"dlogits": _distill_gradient(s, s["logits"].float() / s["temperature"], s["lse"], p, some, at)}


def _attn_scores(s):
    """q, k, v in 32 bits as [heads, tokens, dim], k and v repeated for their group of heads, and the masked scores."""
    t, h = s["q"].shape[:2]
    group = h // s["k"].shape[1]
    q = s["q"].float().transpose(0, 1)
    k, v = (s[n].float().transpose(0, 1).repeat_interleave(group, 0) for n in ("k", "v"))
    at = torch.arange(t, device="cuda")
    seq = torch.searchsorted(s["cu_seqlens"][1:].long(), at, right=True)
    seen = (seq[:, None] == seq[None, :]) & (at[:, None] >= at[None, :])
    scores = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
    return q, k, v, scores.masked_fill_(~seen, float("-inf"))


def _attn_forward(s):
    q, k, v, scores = _attn_scores(s)
    top = scores.amax(2, keepdim=True)
    e = torch.exp(scores - top)
    total = e.sum(2, keepdim=True)
    out = torch.matmul(e, v) / total
    return {"out": out.transpose(0, 1).to(s["q"].dtype).contiguous(), "lse": (top + torch.log(total))[:, :, 0]}


def _attn_backward(s):
    q, k, v, scores = _attn_scores(s)
    t, h, d = s["q"].shape
    kv = s["k"].shape[1]
    p = torch.exp(scores - s["lse"][:, :, None])
    do = s["dout"].float().transpose(0, 1)
    dv = torch.matmul(p.transpose(1, 2), do).view(kv, h // kv, t, d).sum(1)
    dp = torch.matmul(do, v.transpose(1, 2))
    ds = p * (dp - (do * s["out"].float().transpose(0, 1)).sum(2, keepdim=True)) * s["scale"]
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(1, 2), q).view(kv, h // kv, t, d).sum(1)
    return {n: x.transpose(0, 1).to(s["q"].dtype) for n, x in (("dq", dq), ("dk", dk), ("dv", dv))}


_PLAIN = {("ln", "forward"): _ln_forward, ("ln", "backward"): _ln_backward,
          ("distill", "forward"): _distill_forward, ("distill", "step"): _distill_forward,
          ("distill", "backward"): _distill_backward,
          ("attn", "forward"): _attn_forward, ("attn", "backward"): _attn_backward}


# ---- the library's calls -------------------------------------------------------------


def _own(s):
    from allreduce_gradient_reduction_gb300 import binding as ar
    op, direction = s["op"], s["direction"]
    if op == "ln":
        if direction == "forward":
            ar.check(ar.ar_layer_norm(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], eps=s["eps"]))
            return {n: s[n] for n in ("y", "mean", "rstd")}
        if "workspace" not in s:
            s["workspace"] = torch.empty(ar.ar_layer_norm_workspace_bytes(*s["x"].shape), device="cuda",
                                         dtype=torch.uint8)
        ar.check(ar.ar_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"],
                                           s["dbias"], s["workspace"]))
        return {n: s[n] for n in ("dx", "dweight", "dbias")}
    if op == "distill":
        if direction == "backward":
            ar.check(ar.ar_distill_loss_backward(s["logits"], s["index"], s["value"], s["lse"], s["scale"],
                                                 s["dlogits"], temperature=s["temperature"]))
            return {"dlogits": s["dlogits"]}
        dlogits = s.get("dlogits")
        ar.check(ar.ar_distill_loss(s["logits"], s["index"], s["value"], s["loss"], s["lse"], scale=s["scale"],
                                    dlogits=dlogits, temperature=s["temperature"]))
        return {n: s[n] for n in ("loss", "lse", "dlogits") if n in s}
    if direction == "forward":
        ar.check(ar.ar_attention(s["q"], s["k"], s["v"], s["cu_seqlens"], s["out"], s["lse"], scale=s["scale"]))
        return {n: s[n] for n in ("out", "lse")}
    if s["workspace"] is None:
        t, h, d = s["q"].shape
        s["workspace"] = torch.empty(ar.ar_attention_workspace_bytes(t, h, s["k"].shape[1], d), device="cuda",
                                     dtype=torch.uint8)
    ar.check(ar.ar_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["cu_seqlens"], s["dq"],
                                      s["dk"], s["dv"], s["workspace"], scale=s["scale"]))
    return {n: s[n] for n in ("dq", "dk", "dv")}


def run(state):
    return _own(state) if own else _PLAIN[state["op"], state["direction"]](state)


# ---- the definitions in 64 bits -------------------------------------------------------


def _blocks(rows, cols):
    step = max(1, 100000000 // max(1, cols))
    return [slice(a, min(rows, a + step)) for a in range(0, rows, step)]


def _exact_ln(case, s):
    rows, cols = s["x"].shape
    w, b = s["weight"].double(), s["bias"].double()
    parts = []
    dw, db = torch.zeros_like(w), torch.zeros_like(w)
    for at in _blocks(rows, cols):
        x = s["x"][at].double()
        if case["direction"] == "forward":
            var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
            parts.append(((x - mean) / torch.sqrt(var + s["eps"]) * w + b, mean[:, 0], (var + s["eps"])[:, 0] ** -0.5))
        else:
            rstd, dy = s["rstd"][at].double()[:, None], s["dy"][at].double()
            xh = (x - s["mean"][at].double()[:, None]) * rstd
            dw += torch.einsum("rc,rc->c", dy, xh)
            db += dy.sum(0)
            dxh = dy * w
            m1, m2 = dxh.sum(1, keepdim=True) / cols, torch.einsum("rc,rc->r", dxh, xh)[:, None] / cols
            parts.append((rstd * (dxh - m1 - m2 * xh),))
    whole = [torch.cat(p) for p in zip(*parts)]
    return dict(zip(("y", "mean", "rstd"), whole)) if case["direction"] == "forward" else {
        "dx": whole[0], "dweight": dw, "dbias": db}


def _exact_distill(case, s):
    rows, vocab = s["logits"].shape
    tau = float(s["temperature"])
    parts = []
    for at in _blocks(rows, vocab):
        z = s["logits"][at].double() / tau
        idx, val = s["index"][at].long(), s["value"][at].double() / tau
        val[idx < 0] = -math.inf
        teacher = torch.nan_to_num(torch.softmax(val, 1))  # a row without entries: 0/0
        target = torch.zeros_like(z).scatter_add_(1, idx.clamp(min=0), teacher)
        # the lse that a backward call is given is an input; it is the definition's own to within its rounding
        lse = s["lse"][at].double() if case["direction"] == "backward" else torch.logsumexp(z, 1)
        out = {}
        if case["direction"] != "backward":
            logq = torch.gather(z, 1, idx.clamp(min=0)) - lse[:, None]
            out["loss"] = tau * tau * (torch.xlogy(teacher, teacher) - torch.where(teacher > 0, teacher * logq, 0)).sum(1)
            out["lse"] = lse
        if case["direction"] != "forward":
            any_entry = (idx >= 0).any(1, keepdim=True)
            grad = (torch.exp(z - lse[:, None]) - target) * (tau * s["scale"][at].double())[:, None]
            out["dlogits"] = grad * any_entry
        parts.append(out)
    return {n: torch.cat([p[n] for p in parts]) for n in parts[0]}


def _exact_attn(case, s):
    t, h, d = s["q"].shape
    kv = s["k"].shape[1]
    group = h // kv
    forward = case["direction"] == "forward"
    big = {"device": "cuda", "dtype": torch.float64}
    if forward:
        r = {"out": torch.zeros(t, h, d, **big), "lse": torch.zeros(h, t, **big)}
    else:
        r = {"dq": torch.zeros(t, h, d, **big), "dk": torch.zeros(t, kv, d, **big), "dv": torch.zeros(t, kv, d, **big)}
    start = 0
    for n in _lengths(case):
        at = slice(start, start + n)
        start += n
        mask = torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1)
        for j in range(h if n else 0):
            q, k, v = s["q"][at, j].double(), s["k"][at, j // group].double(), s["v"][at, j // group].double()
            a = (q @ k.T * s["scale"]).masked_fill(mask, -math.inf)
            if forward:
                r["lse"][j, at] = torch.logsumexp(a, 1)
                r["out"][at, j] = torch.softmax(a, 1) @ v
                continue
            p = torch.exp(a - s["lse"][j, at].double()[:, None])
            do, o = s["dout"][at, j].double(), s["out"][at, j].double()
            r["dv"][at, j // group] += p.T @ do
            da = p * (do @ v.T - (do * o).sum(1)[:, None]) * s["scale"]
            r["dq"][at, j] = da @ k
            r["dk"][at, j // group] += da.T @ q
    return r


def exact(case, seed):
    s = prepare(case, seed)
    return {"ln": _exact_ln, "distill": _exact_distill, "attn": _exact_attn}[case["op"]](case, s)
