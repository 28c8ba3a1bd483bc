"""Gated codes of very negative gates: silu(gate) x in 64 bits against the
codes. The error of silu(gate) x is that of the header, 2^-19 + |gate| 2^-23 of
the value, and a step of the smallest subnormal."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -149
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rows(cols, dtype):
    """Gates and values; fp16 holds values up to 65504 only."""
    big = min(3e38, torch.finfo(dtype).max)
    g = torch.Generator().manual_seed(cols)
    between = lambda lo, hi: lo + (hi - lo) * torch.rand(cols, generator=g)
    sign = (torch.rand(cols, generator=g) < 0.5) * 2.0 - 1
    gates = [between(-90, -85), torch.full((cols,), -89.0), between(-160, -60), between(-200, -90), between(-84, -82),
             between(-110, -80), torch.full((cols,), -300.0), torch.full((cols,), -torch.finfo(dtype).max), between(-4, 4)]
    values = [torch.ones(cols), torch.full((cols,), big / 30), sign * big / 30, sign * big, sign, sign, sign * big,
              sign * big, sign]
    return torch.stack(gates).to(dtype), torch.stack(values).to(dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cols", [1, 77, 500, 4096, 14336, 30001])
def test_very_negative_gates(cols, dtype):
    from mxfp4_quantized_gemm_amd.int8 import int8_quantize
    gate, x = rows(cols, TYPES[dtype])
    codes, scales = int8_quantize(x.cuda(), gate=gate.cuda())
    g, u = gate.double(), x.double()
    v = g / (1 + torch.exp(-g)) * u
    err = v.abs() * (2.0 ** -19 + g.abs() * 2.0 ** -23 + 4 * U) + TINY
    s = scales.cpu().double()[:, None]
    a = v.abs().amax(1, keepdim=True)
    assert torch.isfinite(s).all()
    assert ((s - a / 127).abs() <= err.amax(1, keepdim=True) / 127 + 2 * U * a / 127 + TINY).all()
    got = codes.cpu()[:, :cols].double() * s
    # the scale of a row of the smallest values is itself off by up to a step
    assert ((got - v).abs() <= s * (0.5 + 127 * 4 * U) + err + 127 * TINY).all()
    # gates of -89 with values near the top: -89 e^-89 x is far above the smallest number in 16 bits with 8 exponent bits
    if dtype != "fp16":
        assert (codes[1, :cols] == -127).all() and float(scales[1]) > 1e-3
    assert not codes[6].any() and scales[6] == 0 and not codes[7].any() and scales[7] == 0


def test_gate_of_minus_infinity():
    """As an infinity or a NaN anywhere in a row."""
    from mxfp4_quantized_gemm_amd.int8 import int8_quantize
    x, g = torch.ones(3, 64), torch.ones(3, 64)
    g[0, 5], g[1, 5], x[1, 5] = float("-inf"), -200.0, float("inf")
    codes, scales = int8_quantize(x.cuda(), gate=g.cuda())
    assert torch.isnan(scales[:2]).all() and not codes[:2].any()
    assert torch.isfinite(scales[2])
