"""torch.autograd.Function wrappers around the C-ABI calls, so the operators can
sit inside a PyTorch training graph.  Every forward and backward runs in
libgbln's kernels (through the functions of this package); nothing here
computes anything itself.

* ``rms_norm(x, weight, eps, residual=None)`` -> ``y`` or ``(y, h)``: RMSNorm with
  the fused residual add.  With a residual, ``h = x + residual`` (the
  residual-stream output) is returned as well, and its gradient enters the
  backward pass as ``dresidual_out``; x and residual get the same gradient.
  The weight gradient comes from the two-pass fixed-order reduction (float32,
  cast to the weight's dtype).
* ``rotary(q, k, positions, cos_sin)`` -> ``(q', k')``: RoPE on Q and K
  (rotate-half pairing); the backward pass is the inverse rotation.
* ``swiglu(gate, up)`` -> ``silu(gate) * up``.

``rms_norm`` and ``swiglu`` take ``checkpoint="int8"`` or ``"e4m3"``: what the backward
pass needs of the input is then kept in 8 bits (one float32 scale per 128 values
of a row, 1.03 bytes per value) instead of in the input's dtype, and the backward
kernels read the codes.  The outputs are those without it (``rms_norm``'s up to the
float32 rounding of a row's sum); the gradients are those of the 8-bit values.
Memory is saved where nothing else keeps the input: the normalised tensor where the
residual stream moves on, gate and up always.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (glu_bwd_ckpt8, glu_fwd_ckpt8, rmsnorm_bwd, rmsnorm_bwd_ckpt8, rmsnorm_dw_finalize,
               rmsnorm_fwd, rmsnorm_fwd_ckpt8, rope_bwd, rope_fwd, swiglu_bwd, swiglu_fwd)


def _c(t):
    return None if t is None else t.contiguous()


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        y, h, rstd = rmsnorm_fwd(x.contiguous(), weight.contiguous(), eps, _c(residual))
        ctx.save_for_backward(h, weight, rstd)
        ctx.has_residual = residual is not None
        if residual is None:
            return y
        return y, h

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        dx, part, P = rmsnorm_bwd(dy.contiguous(), h, weight, rstd, _c(dh))
        dw = rmsnorm_dw_finalize(part, P).to(weight.dtype)
        return dx, (dx if ctx.has_residual else None), dw, None


class _RMSNormCkpt8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, fmt):
        ctx.set_materialize_grads(False)
        weight = weight.contiguous()
        y, h, rstd, h8, scale = rmsnorm_fwd_ckpt8(x.contiguous(), weight, eps, _c(residual), fmt=fmt)
        ctx.save_for_backward(h8, scale, weight, rstd)
        if residual is None:
            return y
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h8, scale, weight, rstd = ctx.saved_tensors
        if dy is None:  # only the residual stream was used
            return dh, dh, None, None, None
        dx, part, P = rmsnorm_bwd_ckpt8(dy.contiguous(), h8, scale, weight, rstd, _c(dh))
        dw = rmsnorm_dw_finalize(part, P).to(weight.dtype)
        return dx, (dx if ctx.needs_input_grad[1] else None), dw, None, None


def rms_norm(x, weight, eps, residual=None, checkpoint=None):
    if checkpoint is None:
        return _RMSNorm.apply(x, residual, weight, float(eps))
    return _RMSNormCkpt8.apply(x, residual, weight, float(eps), checkpoint)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, cos_sin):
        ctx.save_for_backward(positions, cos_sin)
        return rope_fwd(q.contiguous(), k.contiguous(), positions, cos_sin)

    @staticmethod
    def backward(ctx, dq, dk):
        positions, cos_sin = ctx.saved_tensors
        dqi, dki = rope_bwd(dq.contiguous(), dk.contiguous(), positions, cos_sin)
        return dqi, dki, None, None


def rotary(q, k, positions, cos_sin):
    return _Rotary.apply(q, k, positions, cos_sin)


class _SwiGLU(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up):
        gate, up = gate.contiguous(), up.contiguous()
        ctx.save_for_backward(gate, up)
        return swiglu_fwd(gate, up)

    @staticmethod
    def backward(ctx, dout):
        gate, up = ctx.saved_tensors
        return swiglu_bwd(dout.contiguous(), gate, up)


class _SwiGLUCkpt8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up, fmt):
        if gate.shape != up.shape or gate.dtype != up.dtype:
            raise ValueError("gate and up must have the same shape and dtype")
        g, u = (t.flatten(0, -2) if t.dim() > 1 else t.unsqueeze(0) for t in (gate, up))
        # rows of a packed projection output are taken as they lie
        g, u = (t if t.stride(1) == 1 and t.stride(0) >= t.shape[1] else t.contiguous() for t in (g, u))
        out, *saved = glu_fwd_ckpt8(g, u, "silu", fmt=fmt)
        ctx.save_for_backward(*saved)
        return out.view(gate.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        saved = ctx.saved_tensors
        dgate, dup = glu_bwd_ckpt8(dout.contiguous().view(saved[0].shape), *saved, "silu")
        return dgate.view(dout.shape), dup.view(dout.shape), None


def swiglu(gate, up, checkpoint=None):
    if checkpoint is None:
        return _SwiGLU.apply(gate, up)
    return _SwiGLUCkpt8.apply(gate, up, checkpoint)
