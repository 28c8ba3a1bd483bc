"""RMS norm with the residual's addition, in front of a linear layer.

    h = x + residual (held in their type),  y = h / sqrt(mean(h^2) + eps) * weight

``rms_norm`` returns y in the input's type, with gradients (the norm in front
of an MXFP4Linear in training); ``rms_norm_int8`` returns it as the int8
operand of ``int8_gemm`` (serving). Inputs are float32, bfloat16 or float16
of shape [..., cols], cols up to 32768; the weight [cols] is of the same type
or float32. Marshalling only: every step runs in the library's kernels.
"""
from __future__ import annotations

import torch

from . import (mxfp4_rmsnorm, mxfp4_rmsnorm_bwd, mxfp4_rmsnorm_bwd_workspace_bytes,
               mxfp4_rmsnorm_int8)


def _rows(t):
    """t as [rows][cols] with a unit column stride (a view where it has one)."""
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1])
    if t.stride(1) != 1 or t.stride(0) < t.size(1):
        t = t.contiguous()
    return t


def _forward(x, residual, weight, eps, want_rstd):
    h = None if residual is None else torch.empty_like(x, memory_format=torch.contiguous_format)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    rstd = torch.empty(x.size(0), dtype=torch.float32, device=x.device) if want_rstd else None
    mxfp4_rmsnorm(x, residual, weight, eps, h, y, rstd)
    return y, h, rstd


class RMSNormFunction(torch.autograd.Function):
    """(y, h) of 2-D rows; y alone without a residual."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        ctx.set_materialize_grads(False)
        y, h, rstd = _forward(x, residual, weight, eps, True)
        ctx.save_for_backward(x if h is None else h, weight, rstd)
        ctx.added = h is not None
        return (y, h) if ctx.added else y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        want_w = weight is not None and ctx.needs_input_grad[2]
        if dy is None:  # y was not used
            return dh, dh if ctx.added else None, torch.zeros_like(weight) if want_w else None, None
        dy = _rows(dy)
        dh = None if dh is None else _rows(dh)
        dx = torch.empty_like(h, memory_format=torch.contiguous_format)
        dw = ws = None
        if want_w:
            dw = torch.empty_like(weight)
            ws = torch.empty(mxfp4_rmsnorm_bwd_workspace_bytes(*h.shape), dtype=torch.uint8,
                             device=h.device)
        mxfp4_rmsnorm_bwd(dy, dh, h, weight, rstd, dx, dw, ws)
        return dx, dx if ctx.added else None, dw, None


def _check(x, weight, residual):
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual must be {list(x.shape)}, got {list(residual.shape)}")
    if weight is not None and weight.dim() != 1:
        raise ValueError("weight must have one dimension")


def rms_norm(x, weight=None, eps=1e-5, residual=None):
    """y, or (y, h) with a residual; differentiable in x, residual and weight."""
    _check(x, weight, residual)
    x2 = _rows(x)
    r2 = None if residual is None else _rows(residual)
    if torch.is_grad_enabled() and (x.requires_grad or (residual is not None and residual.requires_grad)
                                    or (weight is not None and weight.requires_grad)):
        out = RMSNormFunction.apply(x2, r2, weight, eps)
        y, h = out if residual is not None else (out, None)
    else:
        y, h, _ = _forward(x2, r2, weight, eps, False)
    if x.dim() != 2:
        y = y.view(x.shape)
        h = None if h is None else h.view(x.shape)
    return y if residual is None else (y, h)


def rms_norm_int8(x, weight=None, eps=1e-5, residual=None):
    """(codes, scales), or (codes, scales, h) with a residual; no gradient.

    codes int8 [rows][cols rounded up to 128] with zero codes past cols,
    scales float32 [rows]; the leading dimensions of x are flattened.
    """
    _check(x, weight, residual)
    x2 = _rows(x)
    r2 = None if residual is None else _rows(residual)
    rows, cols = x2.shape
    codes = torch.empty(rows, (cols + 127) // 128 * 128, dtype=torch.int8, device=x.device)
    scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    h = None if r2 is None else torch.empty_like(x2, memory_format=torch.contiguous_format)
    mxfp4_rmsnorm_int8(x2, r2, weight, eps, h, codes, scales)
    return (codes, scales) if h is None else (codes, scales, h.view(x.shape))


class RMSNorm(torch.nn.Module):
    """RMS norm over the last dimension with a weight; ``forward(x, residual)``
    returns (y, x + residual), ``forward(x)`` y."""

    def __init__(self, features, eps=1e-5, dtype=torch.bfloat16, device=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(features, dtype=dtype, device=device))

    def forward(self, x, residual=None):
        return rms_norm(x, self.weight, self.eps, residual)
