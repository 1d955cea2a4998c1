"""The sequence-layer operators under torch's autograd: what a call of `Seq` records for tensors that require
gradients.  The gradients are those of the handle's own backward calls, on the handle that made the outputs."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import seq as binding


def _unused(name, *grads, which="only the operator's first output does"):
    if any(g is not None for g in grads):
        raise RuntimeError(f"{name} carries no gradients: {which}")


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


class ResNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, seq, x, o, w1, b1, z, act, c, w2, b2, kind, after, eps):
        y, h, stats = seq.resnorm(x, o, w1, b1, z, act, c, w2, b2, kind, after, eps)
        ctx.seq, ctx.options = seq, (act, kind, after)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(y, o, stats, w1, b1, z, c, w2, b2)
        return y, h, stats

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh, dstats):
        _unused("resnorm: stats", dstats, which="its first two outputs do")
        if dy is None and dh is None:
            return (None,) * 13
        y, o, stats, w1, b1, z, c, w2, b2 = ctx.saved_tensors
        act, kind, after = ctx.options
        dh = torch.zeros(y.shape, dtype=y.dtype, device=y.device) if dh is None else dh.contiguous()
        dy = None if dy is None else dy.contiguous()
        needs = ctx.needs_input_grad
        dx, do = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (y, o))
        dz = torch.empty(z.shape, dtype=z.dtype, device=z.device) if needs[5] else None
        dw1, db1, dc, dw2, db2 = (torch.empty(t.shape, dtype=t.dtype, device=t.device) if need else None
                                  for t, need in ((w1, needs[3]), (b1, needs[4]), (c, needs[7]), (w2, needs[8]), (b2, needs[9])))
        ctx.seq._on_stream()
        binding.zsolve_resnorm_bwd(ctx.seq.seq, dh, dy, y, o, stats, w1, b1, z, act, c, w2, b2, kind, after, dx, do, dz, dw1, db1, dc,
                                   dw2, db2)
        return None, dx, do, dw1, db1, dz, None, dc, dw2, db2, None, None, None


class Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, seq, x, w, b, act, r, keep):
        y, z = seq.linear(x, w, b, act, r, keep=True) if keep or act != "none" else (seq.linear(x, w, b, act, r), None)
        ctx.seq, ctx.act, ctx.added = seq, act, None if r is None else r.shape
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
        return None, dx, dw, db, None, dy.reshape(ctx.added) if needs[5] else None, None


class Glu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, seq, x, wg, wu, bg, bu, act, keep):
        y, zg, zu = seq.glu(x, wg, wu, bg, bu, act, keep=True)
        ctx.seq, ctx.act = seq, act
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, wg, wu, zg, zu)
        return (y, zg, zu) if keep else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dzg=None, dzu=None):
        _unused("glu: zg and zu", dzg, dzu)
        if dy is None:
            return (None,) * 8
        x, wg, wu, zg, zu = ctx.saved_tensors
        needs = ctx.needs_input_grad[1:6]
        shapes = (x.shape, wg.shape, wu.shape, wg.shape[:1], wu.shape[:1])
        grads = [torch.empty(n, dtype=x.dtype, device=x.device) if need else None for n, need in zip(shapes, needs)]
        if any(needs):
            ctx.seq._on_stream()
            binding.zsolve_glu_bwd(ctx.seq.seq, dy.contiguous(), x, wg, wu, ctx.act, zg, zu, *grads)
        return (None, *grads, None, None)


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
        return (None, *grads, ds0.view(s0.shape) if s0 is not None else None, None, None)


class Decay(torch.autograd.Function):
    @staticmethod
    def forward(ctx, seq, q, k, v, g, s0, offsets, scale):
        o, s = seq.decay(q, k, v, g, s0, offsets, scale)
        ctx.seq, ctx.scale = seq, scale
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, v, g, s0, offsets)
        return o, s

    @staticmethod
    @once_differentiable
    def backward(ctx, do, ds):
        if do is None and ds is None:
            return (None,) * 8
        q, k, v, g, s0, offsets = ctx.saved_tensors
        do = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if do is None else do.contiguous()
        ds = None if ds is None else ds.contiguous()
        *grads, ds0 = ctx.seq.decay_bwd(do, q, k, v, g, s0, ds, offsets, ctx.scale)
        return (None, *grads, ds0.view(s0.shape) if s0 is not None else None, None, None)


class DecayStep(torch.autograd.Function):
    @staticmethod
    def forward(ctx, seq, q, k, v, g, s, s_out, scale):
        o, s_out = seq.decay_step(q, k, v, g, s, s_out, scale)
        ctx.mark_dirty(s_out)
        return o, s_out

    @staticmethod
    def backward(ctx, do, ds):
        raise RuntimeError("decay_step carries no gradients: train with decay")


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
