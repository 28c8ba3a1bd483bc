"""RMS norm with the residual's addition, in front of a linear layer.

    h = x + residual (held in their type),  y = h / sqrt(mean(h^2) + eps) * weight

``rms_norm`` returns y in the input's type, with gradients (the norm in front
of an MXFP4Linear in training); ``rms_norm_int8`` returns it as the int8
operand of ``int8_gemm`` (serving). Inputs are float32, bfloat16 or float16
of shape [..., cols], cols up to 32768, with any strides; the weight [cols] is
of the same type or float32. Marshalling only: every step runs in the
library's kernels.
"""
from __future__ import annotations

import torch

from ._load import ops


def rms_norm(x, weight=None, eps=1e-5, residual=None):
    """y, or (y, h) with a residual; differentiable once in x, residual and weight,
    in reverse mode (forward-mode tangents are refused)."""
    return ops.rms_norm(x, weight, eps, residual)


def rms_norm_int8(x, weight=None, eps=1e-5, residual=None):
    """(codes, scales), or (codes, scales, h) with a residual; no gradient.

    codes int8 [rows][cols rounded up to 128] with zero codes past cols,
    scales float32 [rows]; the leading dimensions of x are flattened.
    """
    return ops.rms_norm_int8(x, weight, eps, residual)


class RMSNorm(torch.nn.Module):
    """RMS norm over the last dimension with a weight; ``forward(x, residual)``
    returns (y, x + residual), ``forward(x)`` y."""

    def __init__(self, features, eps=1e-5, dtype=torch.bfloat16, device=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(features, dtype=dtype, device=device))

    def forward(self, x, residual=None):
        return ops.rms_norm(x, self.weight, self.eps, residual)
