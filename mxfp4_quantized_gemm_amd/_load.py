"""The torch binding of the norm, 8-bit and attention operators. Without it they raise:
there is no fallback."""
import torch  # noqa: F401  (its libraries come first)

try:
    from . import _ops as ops
except ImportError as e:
    raise RuntimeError("_ops.so is missing or does not load: build it with "
                       "`python -m mxfp4_quantized_gemm_amd.build`") from e
