"""The training-step operators together: a small decoder of the GPT-2 kind
learns from a teacher's top logits, data-parallel over simulated ranks.

    python -m allreduce_gradient_reduction_gb300.distill_step [--ranks 2] [--steps 5] ...

Every rank has its own copy of the parameters and its own batch of packed
sequences.  A step is each rank's forward and backward pass (the layer norms,
the attention and the loss are the library's, matrix products and the rest
PyTorch's), ar_bucketed_allreduce of all ranks' gradients, and the same plain
update on every rank; the copies stay equal bit for bit.

layer_norm, packed_attention and distill_loss are the operators as PyTorch
functions with gradients, for use in other models as well.  The gradients have
none of their own: asking for second derivatives raises.
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
        raise RuntimeError("the gradients of layer_norm, packed_attention and distill_loss have no derivative: "
                           "second derivatives through them are not available")


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
        ar.check(ar.ar_attention_backward(dout.contiguous(), q, k, v, out, lse, cu_seqlens, dq, dk, dv, workspace),
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


def make_parameters(layers, width, vocab, positions, seed=0, device="cuda"):
    """name: f32 tensor, GPT-2's names and shapes (weights as [in, out])."""
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    shapes = {"wte": (vocab, width), "wpe": (positions, width), "ln_f.weight": (width,), "ln_f.bias": (width,)}
    for i in range(layers):
        for name, shape in (("ln_1.weight", (width,)), ("ln_1.bias", (width,)), ("c_attn.weight", (width, 3 * width)),
                            ("c_attn.bias", (3 * width,)), ("c_proj.weight", (width, width)), ("c_proj.bias", (width,)),
                            ("ln_2.weight", (width,)), ("ln_2.bias", (width,)), ("c_fc.weight", (width, 4 * width)),
                            ("c_fc.bias", (4 * width,)), ("mlp.c_proj.weight", (4 * width, width)),
                            ("mlp.c_proj.bias", (width,))):
            shapes[f"h.{i}.{name}"] = shape
    out = {}
    for name, shape in shapes.items():
        if name.endswith("bias"):
            t = torch.zeros(shape)
        elif ".ln_" in name or name.startswith("ln_"):
            t = torch.ones(shape)
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

    x = (p["wte"][tokens] + p["wpe"][positions]).to(dtype)
    for i in range(layers):
        h = f"h.{i}."
        qkv = linear(norm(x, p[h + "ln_1.weight"], p[h + "ln_1.bias"]), h + "c_attn")
        q, k, v = (t.unflatten(1, (heads, width // heads)) for t in qkv.split(width, 1))
        x = x + linear(attention(q, k, v, cu_seqlens).flatten(1), h + "c_proj")
        y = norm(x, p[h + "ln_2.weight"], p[h + "ln_2.bias"])
        x = x + linear(F.gelu(linear(y, h + "c_fc"), approximate="tanh"), h + "mlp.c_proj")
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
        temperature=2.0, rate=0.5):
    """The ranks' parameters after `steps` steps, and each step's losses."""
    models = [make_parameters(layers, width, vocab, max(lengths)) for _ in range(ranks)]
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
    models, losses = run(**vars(parser.parse_args()))
    for n, each in enumerate(losses):
        print(f"step {n}: mean loss of each rank " + " ".join(f"{x:.4f}" for x in each))
    same = all(torch.equal(a, b) for m in models[1:] for a, b in zip(models[0].values(), m.values()))
    print("the ranks' parameters are " + ("equal bit for bit" if same else "NOT equal"))
    return 0 if same else 1


if __name__ == "__main__":
    raise SystemExit(main())
