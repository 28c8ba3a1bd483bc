"""Linear layers held in 8 bits: int8 codes with a scale for each token and
each output channel, for layers and tokens that the MXFP4 products do not
serve (any number of rows from one, any width).

    codes, scales = int8_quantize(x)          one scale a row, a / 127
    c = int8_gemm(a, a_scales, b, b_scales)   (sum_k a b, exact) * scales
    y = int8_linear(x, w, w_scales)           both

An operand is int8 [rows][pitch]: the pitch is the width rounded up to a
multiple of 128, with zero codes past the width, which a product runs over.
Inference only (the codes have no gradient). Marshalling only: every step
runs in the library's kernels.
"""
from __future__ import annotations

import torch

from . import mxfp4_int8_gemm, mxfp4_int8_gemm_workspace_bytes, mxfp4_int8_quantize
from .norm import _rows, rms_norm_int8


def int8_quantize(x, gate=None):
    """(codes, scales) of the rows of x, or of silu(gate) * x; leading
    dimensions are flattened."""
    if gate is not None and gate.shape != x.shape:
        raise ValueError(f"gate must be {list(x.shape)}, got {list(gate.shape)}")
    x2 = _rows(x)
    rows, cols = x2.shape
    codes = torch.empty(rows, (cols + 127) // 128 * 128, dtype=torch.int8, device=x.device)
    scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    mxfp4_int8_quantize(x2, None if gate is None else _rows(gate), codes, scales)
    return codes, scales


def int8_gemm(a, a_scales, b, b_scales, bias=None, out_dtype=torch.bfloat16):
    """C [M][N] of int8 a [M][K] and b [N][K], fp32 scales [M] and [N], and an
    fp32 bias [N]."""
    M, K = a.shape
    N = b.size(0)
    need = mxfp4_int8_gemm_workspace_bytes(M, N, K)
    ws = torch.empty(need, dtype=torch.uint8, device=a.device) if need else None
    c = torch.empty(M, N, dtype=out_dtype, device=a.device)
    mxfp4_int8_gemm(a, a_scales, b, b_scales, bias, c, ws)
    return c


def _product(codes, scales, cols, w, w_scales, bias, out_dtype):
    """The product of quantized rows of `cols` values with a weight that is
    padded as they are, or that has just `cols` columns."""
    if w.dim() != 2 or w.size(1) not in (cols, codes.size(1)):
        raise ValueError(f"weight codes must have {cols} or {codes.size(1)} columns, got {list(w.shape)}")
    if w.size(1) != codes.size(1):
        codes = codes[:, :cols]
    return int8_gemm(codes, scales, w, w_scales, bias, out_dtype)


def int8_linear(x, w, w_scales, bias=None, out_dtype=None):
    """x [..., K] quantized row by row, times w^T; out_dtype: x's type."""
    codes, scales = int8_quantize(x)
    y = _product(codes, scales, x.shape[-1], w, w_scales, bias, out_dtype or x.dtype)
    return y if x.dim() == 2 else y.view(*x.shape[:-1], w.size(0))


def int8_mlp(x, norm_weight, eps, gate_up, gate_up_scales, down, down_scales, residual=None):
    """A feed-forward block in 8 bits: norm (of x + residual), gate and up
    rows in one product (gate_up [2 F][K]: the gate's F rows first), silu(gate)
    * up quantized in one pass, down product. Returns (y, h), h = x + residual
    (x itself without a residual); the caller adds y to h, or hands both to
    the next block's norm."""
    out = rms_norm_int8(x, norm_weight, eps, residual)
    codes, scales = out[0], out[1]
    gu = _product(codes, scales, x.shape[-1], gate_up, gate_up_scales, None, x.dtype)
    F = gu.size(1) // 2
    codes, scales = int8_quantize(gu[:, F:], gate=gu[:, :F])
    y = _product(codes, scales, F, down, down_scales, None, x.dtype)
    return y.view(*x.shape[:-1], y.size(1)), (x if residual is None else out[2])


class Int8Linear(torch.nn.Module):
    """Linear layer with int8 weight codes [out][in rounded up to 128], a
    scale for each output channel and an optional fp32 bias (buffers: this
    layer is not trained)."""

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
        """From a weight [out][in] in GPU memory (a Linear's or MXFP4Linear's)."""
        layer = cls(weight.size(1), weight.size(0), bias is not None, weight.device)
        layer.weight, layer.scales = int8_quantize(weight.detach())
        if bias is not None:
            layer.bias = bias.detach().float()
        return layer

    def forward(self, x):
        if x.shape[-1] != self.in_features:
            raise ValueError(f"the last dimension must be {self.in_features}, got {x.shape[-1]}")
        return int8_linear(x, self.weight, self.scales, self.bias)
