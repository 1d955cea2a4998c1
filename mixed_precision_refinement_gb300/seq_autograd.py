"""The sequence-layer operators under torch's autograd: what a call of `Seq` records for tensors that require
gradients.  The gradients are those of the handle's own backward calls, on the handle that made the outputs."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import seq as binding


def _unused(name, *grads):
    if any(g is not None for g in grads):
        raise RuntimeError(f"{name} carries no gradients: only the operator's first output does")


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, seq, x, w, b, eps):
        y, mean, rstd = seq.layernorm(x, w, b, eps)
        ctx.seq, ctx.types = seq, (w.dtype if w is not None else None, b.dtype if b is not None else None)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, w, mean, rstd)
        return y, mean, rstd

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dmean, drstd):
        _unused("layernorm: mean and rstd", dmean, drstd)
        if dy is None:
            return (None,) * 5
        x, w, mean, rstd = ctx.saved_tensors
        dx = torch.empty_like(x)
        dw, db = (torch.empty(x.shape[-1], dtype=t, device=x.device) if need else None
                  for t, need in zip(ctx.types, ctx.needs_input_grad[2:4]))
        ctx.seq._on_stream()
        binding.zsolve_layernorm_bwd(ctx.seq.seq, dy.contiguous(), x, mean, rstd, w, dx, dw, db)
        return None, dx, dw, db, None


class Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, seq, x, w, b, act, r, keep):
        y, z = seq.linear(x, w, b, act, r, keep=True) if keep or act != "none" else (seq.linear(x, w, b, act, r), None)
        ctx.seq, ctx.act = seq, act
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, w, z)
        return (y, z) if keep else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dz=None):
        _unused("linear: z", dz)
        if dy is None:
            return (None,) * 7
        x, w, z = ctx.saved_tensors
        needs = ctx.needs_input_grad
        dx = torch.empty_like(x) if needs[1] else None
        dw = torch.empty_like(w) if needs[2] else None
        db = torch.empty(w.shape[:1], dtype=x.dtype, device=x.device) if needs[3] else None
        if any(needs[1:4]):
            ctx.seq._on_stream()
            binding.zsolve_linear_bwd(ctx.seq.seq, dy.contiguous(), x, w, ctx.act, z, dx, dw, db)
        return None, dx, dw, db, None, dy if needs[5] else None, None


class Delta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, seq, q, k, v, g, beta, s0, offsets, scale):
        o, s = seq.delta(q, k, v, g, beta, s0, offsets, scale)
        ctx.seq, ctx.scale = seq, scale
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, v, g, beta, s0, offsets)
        return o, s

    @staticmethod
    @once_differentiable
    def backward(ctx, do, ds):
        if do is None and ds is None:
            return (None,) * 9
        q, k, v, g, beta, s0, offsets = ctx.saved_tensors
        do = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if do is None else do.contiguous()
        ds = None if ds is None else ds.contiguous()
        *grads, ds0 = ctx.seq.delta_bwd(do, q, k, v, g, beta, s0, ds, offsets, ctx.scale)
        return (None, *grads, ds0 if s0 is not None else None, None, None)


class Step(torch.autograd.Function):
    """The token-by-token form, for answering, has no gradients: a backward pass that reaches it is an error."""

    @staticmethod
    def forward(ctx, seq, q, k, v, g, beta, s, s_out, scale):
        o, s_out = seq.delta_step(q, k, v, g, beta, s, s_out, scale)
        ctx.mark_dirty(s_out)
        return o, s_out

    @staticmethod
    def backward(ctx, do, ds):
        raise RuntimeError("delta_step carries no gradients: train with delta")
