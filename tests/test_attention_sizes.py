"""Sizes that attention's workspace functions refuse (no GPU)."""
import pytest

import mxfp4_quantized_gemm_amd as mx


@pytest.mark.parametrize("heads", [-1, -(1 << 63), 1025, 1 << 40, (1 << 63) - 1])
def test_workspace_of_heads_that_the_gradient_refuses(heads):
    size = mx.load_library().mxfp4_qk_norm_rope_bwd_workspace_bytes
    assert size(3, heads, 2, 64) == 0 and size(3, 4, heads, 64) == 0 and size(3, heads, heads, 64) == 0
    assert size(3, 1024, 1024, 64) > 0 and size(3, 0, 0, 64) > 0
