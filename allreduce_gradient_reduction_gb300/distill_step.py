"""The training-step operators together: a small decoder of the GPT-2 kind
learns from a teacher's top logits, data-parallel over simulated ranks.

    python -m allreduce_gradient_reduction_gb300.distill_step [--ranks 2] [--steps 5] ...

Every rank has its own copy of the parameters and its own batch of packed
sequences.  A step is each rank's forward and backward pass (the layer norms,
the attention and the loss are the library's, matrix products and the rest
PyTorch's), ar_bucketed_allreduce of all ranks' gradients, and the same plain
update on every rank; the copies stay equal bit for bit.

--block diff trains another kind of decoder: queries and keys are normalised for
each head and turned by their positions (there is no table of positions),
attention is the difference of two maps with a learned weight for each head, and
the hidden layer's input is kept in 8 bits for the backward pass.

layer_norm, packed_attention, distill_loss, qk_norm_rope, diff_attention and
activation8_linear are the operators as PyTorch functions with gradients, for
use in other models as well.  The gradients have none of their own: asking for
second derivatives raises.
"""
import argparse
import functools

import torch
import torch.nn.functional as F

from . import binding as ar


class _NoSecondDerivative(torch.autograd.Function):
    """Its first `count` tensors, which depend on all of them in a way that is
    not differentiable."""
    @staticmethod
    def forward(ctx, count, *tensors):
        return tuple(t.view_as(t) for t in tensors[:count])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gradients of the library's operators have no derivative: second derivatives through "
                           "them are not available")


def _once(backward):
    """For a Function's backward that is made of calls autograd does not see.
    Where a graph of the gradients is asked for, they are tied to what they
    depend on, so that differentiating them again raises.  (torch's own
    once_differentiable ties them to nothing: autograd.grad with respect to
    the inputs then takes them for constants.)"""
    @functools.wraps(backward)
    def wrapped(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        out = out if isinstance(out, tuple) else (out,)
        made = [t for t in out if t is not None]
        tied = iter(_NoSecondDerivative.apply(len(made), *made, *grads, *ctx.saved_tensors))
        return tuple(None if t is None else next(tied) for t in out)
    return wrapped


def _rows(grad):
    """An upstream gradient as the attention calls take it, which is on a 16-byte
    boundary: a part of a concatenation's gradient begins anywhere."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y = torch.empty_like(x)
        mean, rstd = torch.empty((2, x.shape[0]), dtype=torch.float32, device=x.device)
        ar.check(ar.ar_layer_norm(x, weight, bias, y, mean, rstd, eps), "ar_layer_norm")
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    @_once
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dweight = torch.empty_like(x), torch.empty_like(weight)
        dbias = torch.empty_like(weight) if ctx.has_bias else None
        workspace = torch.empty(ar.ar_layer_norm_workspace_bytes(*x.shape), dtype=torch.uint8, device=x.device)
        ar.check(ar.ar_layer_norm_backward(dy.contiguous(), x, weight, mean, rstd, dx, dweight, dbias, workspace),
                 "ar_layer_norm_backward")
        return dx, dweight, dbias, None


def layer_norm(x, weight, bias, eps=1e-5):
    """x [rows, cols]; weight and bias of x's type or f32, bias may be None."""
    return _LayerNorm.apply(x, weight, bias, eps)


class _PackedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens):
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[1], q.shape[0], dtype=torch.float32, device=q.device)
        ar.check(ar.ar_attention(q, k, v, cu_seqlens, out, lse), "ar_attention")
        ctx.save_for_backward(q, k, v, cu_seqlens, out, lse)
        return out

    @staticmethod
    @_once
    def backward(ctx, dout):
        q, k, v, cu_seqlens, out, lse = ctx.saved_tensors
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        workspace = torch.empty(ar.ar_attention_workspace_bytes(*q.shape[:2], k.shape[1], q.shape[2]),
                                dtype=torch.uint8, device=q.device)
        ar.check(ar.ar_attention_backward(_rows(dout), q, k, v, out, lse, cu_seqlens, dq, dk, dv, workspace),
                 "ar_attention_backward")
        return dq, dk, dv, None


def packed_attention(q, k, v, cu_seqlens):
    """q [tokens, heads, dim], k and v [tokens, kv_heads, dim], bf16 or f16;
    the sequences have to cover every token."""
    return _PackedAttention.apply(q, k, v, cu_seqlens)


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher_index, teacher_logits, temperature):
        loss, lse = torch.empty((2, logits.shape[0]), dtype=torch.float32, device=logits.device)
        ar.check(ar.ar_distill_loss(logits, teacher_index, teacher_logits, loss, lse, temperature=temperature),
                 "ar_distill_loss")
        ctx.save_for_backward(logits, teacher_index, teacher_logits, lse)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @_once
    def backward(ctx, dloss):
        logits, teacher_index, teacher_logits, lse = ctx.saved_tensors
        dlogits = torch.empty_like(logits)
        ar.check(ar.ar_distill_loss_backward(logits, teacher_index, teacher_logits, lse, dloss.contiguous(), dlogits,
                                             temperature=ctx.temperature), "ar_distill_loss_backward")
        return dlogits, None, None, None


def distill_loss(logits, teacher_index, teacher_logits, temperature=1.0):
    """The loss of each row.  Where the mean's gradient is wanted at once,
    ar_distill_loss with dlogits makes both in one pass over the logits."""
    return _DistillLoss.apply(logits, teacher_index, teacher_logits, temperature)


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, how):
        q_out, k_out = (None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k))
        ar.check(ar.ar_qk_norm_rope(q, k, q_weight, k_weight, positions, q_out, k_out, **how), "ar_qk_norm_rope")
        ctx.save_for_backward(q, k, q_weight, k_weight, positions)
        ctx.how = how
        return q_out, k_out

    @staticmethod
    @_once
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, positions = ctx.saved_tensors
        dq, dk = (None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k))
        dq_weight, dk_weight = (None if w is None else torch.empty_like(w) for w in (q_weight, k_weight))
        kv_heads = 0 if k is None else k.shape[1]
        workspace = torch.empty(ar.ar_qk_norm_rope_workspace_bytes(*q.shape[:2], kv_heads, q.shape[2]),
                                dtype=torch.uint8, device=q.device)
        dq_out, dk_out = dq_out.contiguous(), None if k is None else dk_out.contiguous()
        ar.check(ar.ar_qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, dq, dk, dq_weight,
                                             dk_weight, workspace, **ctx.how),
                 "ar_qk_norm_rope_backward")
        return dq, dk, dq_weight, dk_weight, None, None


def qk_norm_rope(q, k, q_weight, k_weight, positions, **how):
    """q [tokens, heads, dim] and k [tokens, kv_heads, dim], each head
    normalised, weighted [dim] (None: not weighted) and turned by its token's
    position (i32).  k may be None, as is its result then.  how:
    ar_qk_norm_rope's rotary_dim, base, frequencies, interleaved and eps."""
    return _QkNormRope.apply(q, k, q_weight, k_weight, positions, how)


class _DiffAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lam, cu_seqlens, how):
        shape = (q.shape[0], lam.shape[0], v.shape[2])
        out, second = (torch.empty(shape, dtype=q.dtype, device=q.device) for _ in range(2))
        lse = torch.empty(q.shape[1], q.shape[0], dtype=torch.float32, device=q.device)
        ar.check(ar.ar_diff_attention(q, k, v, lam, cu_seqlens, out, second, lse, **how), "ar_diff_attention")
        ctx.save_for_backward(q, k, v, lam, cu_seqlens, out, second, lse)
        ctx.how = how
        return out

    @staticmethod
    @_once
    def backward(ctx, dout):
        q, k, v, lam, cu_seqlens, out, second, lse = ctx.saved_tensors
        dq, dk, dv, dlam = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v, lam))
        workspace = torch.empty(ar.ar_diff_attention_workspace_bytes(q.shape[0], lam.shape[0], v.shape[1], q.shape[2],
                                                                     v.shape[2]), dtype=torch.uint8, device=q.device)
        ar.check(ar.ar_diff_attention_backward(_rows(dout), q, k, v, lam, out, second, lse, cu_seqlens, dq, dk,
                                               dv, dlam, workspace, **ctx.how), "ar_diff_attention_backward")
        return dq, dk, dv, dlam, None, None


def diff_attention(q, k, v, lam, cu_seqlens, scale=None):
    """q [tokens, 2 heads, dim], k [tokens, 2 kv_heads, dim], v [tokens,
    kv_heads, value_dim], bf16 or f16; lam [heads] f32; scale None: dim ** -0.5.
    The sequences have to cover every token."""
    return _DiffAttention.apply(q, k, v, lam, cu_seqlens, {} if scale is None else {"scale": scale})


class _Activation8Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, kind):
        rows, cols = x.shape
        blocks = -(-cols // ar.ACTIVATION8_BLOCK)
        y = torch.empty_like(x)
        codes = torch.empty(rows, blocks * ar.ACTIVATION8_BLOCK, dtype=torch.int8, device=x.device)
        scales = torch.empty(rows, blocks, dtype=torch.float32, device=x.device)
        ar.check(ar.ar_activation8(x, y, codes, scales, kind=kind), "ar_activation8")
        ctx.save_for_backward(codes, scales, weight)
        ctx.kind = kind
        ctx.has_bias = bias is not None
        return y @ weight if bias is None else torch.addmm(bias, y, weight)

    @staticmethod
    @_once
    def backward(ctx, dout):
        codes, scales, weight = ctx.saved_tensors
        dy = dout @ weight.t()
        y = torch.empty_like(dy)
        ar.check(ar.ar_activation8_backward(codes, scales, dy, dy, y, kind=ctx.kind), "ar_activation8_backward")
        return dy, y.t() @ dout, dout.sum(0) if ctx.has_bias else None, None


def activation8_linear(x, weight, bias, kind="gelu_tanh"):
    """activation(x) @ weight + bias, all of one type; bias may be None.  Neither x nor the
    activation is kept for the backward pass, but x in 8 bits: gradients are
    those at what the codes stand for, the weight's with the activation made
    again from them."""
    return _Activation8Linear.apply(x, weight, bias, kind)


BLOCKS = ("gpt2", "diff")


def make_parameters(layers, width, vocab, positions, seed=0, device="cuda", block="gpt2", heads=1):
    """name: f32 tensor, GPT-2's names and shapes (weights as [in, out]).
    block "diff", of `heads` heads: weights of the norms of queries and keys and
    of the second maps in the place of a table of positions."""
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    shapes = {"wte": (vocab, width), "wpe": (positions, width), "ln_f.weight": (width,), "ln_f.bias": (width,)}
    if block == "diff":
        del shapes["wpe"]
    for i in range(layers):
        for name, shape in (("ln_1.weight", (width,)), ("ln_1.bias", (width,)), ("c_attn.weight", (width, 3 * width)),
                            ("c_attn.bias", (3 * width,)), ("c_proj.weight", (width, width)), ("c_proj.bias", (width,)),
                            ("ln_2.weight", (width,)), ("ln_2.bias", (width,)), ("c_fc.weight", (width, 4 * width)),
                            ("c_fc.bias", (4 * width,)), ("mlp.c_proj.weight", (4 * width, width)),
                            ("mlp.c_proj.bias", (width,))):
            shapes[f"h.{i}.{name}"] = shape
        if block == "diff":
            for name, n in (("q_norm.weight", width // heads // 2), ("k_norm.weight", width // heads // 2),
                            ("lambda", heads)):
                shapes[f"h.{i}.{name}"] = (n,)
    out = {}
    for name, shape in shapes.items():
        if name.endswith("bias"):
            t = torch.zeros(shape)
        elif ".ln_" in name or name.startswith("ln_") or "_norm." in name:
            t = torch.ones(shape)
        elif name.endswith("lambda"):
            t = torch.full(shape, 0.5)
        else:
            t = torch.randn(shape, generator=g) * 0.05
        out[name] = t.to(device)
    return out


def logits_of(p, tokens, positions, cu_seqlens, heads, dtype=torch.bfloat16, norm=layer_norm, attention=packed_attention):
    """The decoder over one batch of packed sequences: [tokens, vocab].  norm
    and attention may be other implementations of the same functions."""
    layers = sum(name.endswith("ln_1.weight") for name in p)
    width = p["wte"].shape[1]

    def linear(x, name):
        return x @ p[name + ".weight"].to(dtype) + p[name + ".bias"].to(dtype)

    if "wpe" not in p:
        return diff_logits_of(p, tokens, positions, cu_seqlens, heads, dtype, norm)
    x = (p["wte"][tokens] + p["wpe"][positions]).to(dtype)
    for i in range(layers):
        h = f"h.{i}."
        qkv = linear(norm(x, p[h + "ln_1.weight"], p[h + "ln_1.bias"]), h + "c_attn")
        q, k, v = (t.unflatten(1, (heads, width // heads)) for t in qkv.split(width, 1))
        x = x + linear(attention(q, k, v, cu_seqlens).flatten(1), h + "c_proj")
        y = norm(x, p[h + "ln_2.weight"], p[h + "ln_2.bias"])
        x = x + linear(F.gelu(linear(y, h + "c_fc"), approximate="tanh"), h + "mlp.c_proj")
    return norm(x, p["ln_f.weight"], p["ln_f.bias"]) @ p["wte"].to(dtype).t()


def diff_logits_of(p, tokens, positions, cu_seqlens, heads, dtype=torch.bfloat16, norm=layer_norm,
                   prepare=qk_norm_rope, attention=diff_attention, mlp=activation8_linear):
    """The same for parameters of block "diff"; prepare, attention and mlp may
    be other implementations of the same functions."""
    layers = sum(name.endswith("ln_1.weight") for name in p)
    width = p["wte"].shape[1]
    positions = positions.to(torch.int32)

    def weights(name):
        return p[name + ".weight"].to(dtype), p[name + ".bias"].to(dtype)

    def linear(x, name):
        w, b = weights(name)
        return x @ w + b

    x = p["wte"][tokens].to(dtype)
    for i in range(layers):
        h = f"h.{i}."
        qkv = linear(norm(x, p[h + "ln_1.weight"], p[h + "ln_1.bias"]), h + "c_attn")
        q, k, v = (t.unflatten(1, (n, width // n)) for t, n in zip(qkv.split(width, 1), (2 * heads, 2 * heads, heads)))
        q, k = prepare(q, k, p[h + "q_norm.weight"], p[h + "k_norm.weight"], positions)
        x = x + linear(attention(q, k, v, p[h + "lambda"], cu_seqlens).flatten(1), h + "c_proj")
        y = norm(x, p[h + "ln_2.weight"], p[h + "ln_2.bias"])
        x = x + mlp(linear(y, h + "c_fc"), *weights(h + "mlp.c_proj"))
    return norm(x, p["ln_f.weight"], p["ln_f.bias"]) @ p["wte"].to(dtype).t()


def make_batch(lengths, vocab, top, seed, device="cuda"):
    """Random tokens of sequences of these lengths and a teacher's lists."""
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    n = sum(lengths)
    starts = torch.tensor([0] + list(lengths)).cumsum(0)
    batch = {
        "tokens": torch.randint(0, vocab, (n,), generator=g),
        "positions": torch.cat([torch.arange(x) for x in lengths]),
        "cu_seqlens": starts.to(torch.int32),
        "teacher_index": torch.rand(n, vocab, generator=g).topk(top, 1).indices.to(torch.int32),
        "teacher_logits": torch.randn(n, top, generator=g) * 2,
    }
    return {k: t.to(device) for k, t in batch.items()}


def step(ranks, batches, heads, temperature, rate):
    """One step of all ranks; their mean losses before the update."""
    losses, grads = [], []
    for p, b in zip(ranks, batches):
        for t in p.values():
            t.requires_grad_()
        z = logits_of(p, b["tokens"], b["positions"], b["cu_seqlens"], heads)
        loss = distill_loss(z, b["teacher_index"], b["teacher_logits"], temperature).mean()
        grads.append([g.contiguous().view(-1) for g in torch.autograd.grad(loss, list(p.values()))])
        losses.append(loss.detach())
    ar.check(ar.ar_bucketed_allreduce(grads, op="avg"), "ar_bucketed_allreduce")
    with torch.no_grad():
        for p, g in zip(ranks, grads):
            for t, d in zip(p.values(), g):
                t -= rate * d.view_as(t)
    return [x.item() for x in losses]


def run(ranks=2, steps=5, layers=2, heads=4, width=256, vocab=5003, top=32, lengths=(100, 1, 155, 64),
        temperature=2.0, rate=0.5, block="gpt2"):
    """The ranks' parameters after `steps` steps, and each step's losses."""
    models = [make_parameters(layers, width, vocab, max(lengths), block=block, heads=heads) for _ in range(ranks)]
    batches = [make_batch(lengths, vocab, top, 100 + r) for r in range(ranks)]
    losses = [step(models, batches, heads, temperature, rate) for _ in range(steps)]
    rc, status = ar.ar_device_status()
    ar.check(rc, "ar_device_status")
    ar.check(status, "a kernel gave up waiting")
    return models, losses


def main():
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("ranks", 2), ("steps", 5), ("layers", 2), ("heads", 4), ("width", 256), ("vocab", 5003),
                        ("top", 32)):
        parser.add_argument("--" + name, type=int, default=value)
    parser.add_argument("--block", choices=BLOCKS, default=BLOCKS[0])
    models, losses = run(**vars(parser.parse_args()))
    for n, each in enumerate(losses):
        print(f"step {n}: mean loss of each rank " + " ".join(f"{x:.4f}" for x in each))
    same = all(torch.equal(a, b) for m in models[1:] for a, b in zip(models[0].values(), m.values()))
    print("the ranks' parameters are " + ("equal bit for bit" if same else "NOT equal"))
    return 0 if same else 1


if __name__ == "__main__":
    raise SystemExit(main())
