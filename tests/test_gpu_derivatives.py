"""Derivatives that the norm's gradient does not have are refused where they
would arise, in the backward pass."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("use", ["y", "h", "both"])
def test_tangents_of_incoming_gradients(use):
    """Forward over reverse: a factor of y (use "y") or of h carries a tangent."""
    import torch.autograd.forward_ad as fwd
    from mxfp4_quantized_gemm_amd.norm import rms_norm
    x = torch.randn(4, 64, device="cuda").requires_grad_(True)
    y, h = rms_norm(x, None, residual=torch.randn(4, 64, device="cuda"))
    c = torch.randn(4, 64, device="cuda")

    def loss(factor):
        return ((y if use == "y" else h) * factor).sum() + (y.sum() if use == "both" else 0)
    plain, = torch.autograd.grad(loss(c), x, retain_graph=True)
    with fwd.dual_level():
        dual = loss(fwd.make_dual(c, torch.ones_like(c)))
        if use == "h":  # y is not used: h's gradient is x's, with its tangent
            dx, = torch.autograd.grad(dual, x)
            dx, tangent = fwd.unpack_dual(dx)
            assert torch.equal(dx, plain) and torch.equal(tangent, torch.ones_like(c))
        else:
            with pytest.raises(RuntimeError, match="forward-mode"):
                torch.autograd.grad(dual, x)
