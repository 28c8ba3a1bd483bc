"""Linear layers held in 8 bits: int8 codes with a scale for each token and
each output channel, for layers and tokens that the MXFP4 products do not
serve (any number of rows from one, widths that are no multiple of 32).

    codes, scales = int8_quantize(x)          one scale a row, a / 127
    c = int8_gemm(a, a_scales, b, b_scales)   (sum_k a b, exact) * scales
    y = int8_linear(x, w, w_scales)           both

An operand is int8 [rows][pitch]: the pitch is the width rounded up to a
multiple of 128, with zero codes past the width, which a product runs over. (Codes
of the width alone are taken too, by a kernel that is several times slower.)
The quantizers take rows of up to 32768 columns, a product K up to 131071;
wider calls raise.
Inference only: a call in which an input, a scale or the bias requires a gradient
is refused (torch.no_grad() or detached tensors). Marshalling only: every step
runs in the library's kernels.
"""
from __future__ import annotations

import torch

from ._load import ops


def int8_quantize(x, gate=None):
    """(codes, scales) of the rows of x, or of silu(gate) * x; leading
    dimensions are flattened."""
    return ops.int8_quantize(x, gate)


def int8_gemm(a, a_scales, b, b_scales, bias=None, out_dtype=torch.bfloat16):
    """C [M][N] of int8 a [M][K] and b [N][K], fp32 scales [M] and [N], and an
    fp32 bias [N]."""
    return ops.int8_gemm(a, a_scales, b, b_scales, bias, out_dtype)


def int8_linear(x, w, w_scales, bias=None, out_dtype=None):
    """x [..., K] quantized row by row, times w^T; out_dtype: x's type."""
    return ops.int8_linear(x, w, w_scales, bias, out_dtype)


def int8_mlp(x, norm_weight, eps, gate_up, gate_up_scales, down, down_scales, residual=None):
    """A feed-forward block in 8 bits: norm (of x + residual), gate and up
    rows in one product (gate_up [2 F][K]: the gate's F rows first; its result
    is held in x's type), silu(gate) * up quantized in one pass, down product. Returns (y, h), h = x + residual
    (x itself without a residual); the caller adds y to h, or hands both to
    the next block's norm."""
    return ops.int8_mlp(x, norm_weight, eps, gate_up, gate_up_scales, down, down_scales, residual)


class Int8Linear(torch.nn.Module):
    """Linear layer with int8 weight codes [out][in rounded up to 128], a
    scale for each output channel and an optional fp32 bias (buffers: this
    layer is not trained). Casts of a model (bfloat16(), to(dtype), ...) leave
    their types and values as they are."""

    def __init__(self, in_features, out_features, bias=False, device=None):
        super().__init__()
        self.in_features, self.out_features = in_features, out_features
        pitch = (in_features + 127) // 128 * 128
        self.register_buffer("weight", torch.zeros(out_features, pitch, dtype=torch.int8, device=device))
        self.register_buffer("scales", torch.zeros(out_features, dtype=torch.float32, device=device))
        self.register_buffer("bias", torch.zeros(out_features, dtype=torch.float32, device=device)
                             if bias else None)

    @classmethod
    @torch.no_grad()
    def from_weight(cls, weight, bias=None):
        """From a weight [out][in] in GPU memory (a Linear's or MXFP4Linear's) and
        its bias; both are copied."""
        if bias is not None and bias.numel() != weight.size(0):
            raise ValueError(f"bias must hold {weight.size(0)} values, holds {bias.numel()}")
        layer = cls(weight.size(1), weight.size(0), bias is not None, weight.device)
        layer.weight, layer.scales = int8_quantize(weight.detach())
        if bias is not None:
            layer.bias.copy_(bias.reshape(-1))
        return layer

    def _apply(self, fn, recurse=True):
        # Module's casts and moves come through here: take the moves only
        kept = dict(self._buffers)
        super()._apply(fn, recurse)
        for name, b in kept.items():
            if b is not None and self._buffers[name].dtype != b.dtype:
                self._buffers[name] = b.to(self._buffers[name].device)
        return self

    def forward(self, x):
        if x.shape[-1] != self.in_features:
            raise ValueError(f"the last dimension must be {self.in_features}, got {x.shape[-1]}")
        return ops.int8_linear(x, self.weight, self.scales, self.bias, None)
