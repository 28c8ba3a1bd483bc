"""Gradients of qk_norm_rope where queries, keys or both have no head."""
import pytest
import torch

from tests.attention_util import frequencies, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,K,read", [(0, 0, "both"), (0, 0, "k"), (3, 0, "k"), (0, 2, "q"), (3, 0, "both"), (0, 2, "both")])
@pytest.mark.parametrize("norm", [True, False])
def test_gradients_where_no_head_is(H, K, read, norm):
    """Empty gradients of the heads, and zeros for a weight that none of them has met."""
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope
    q, k = (rand((5, n, 64), torch.float32, n + 1).cuda().requires_grad_(True) for n in (H, K))
    w = [(1 + 0.1 * rand((64,), torch.float32, i)).cuda().requires_grad_(True) if norm else None for i in (3, 4)]
    out = qk_norm_rope(q, k, torch.arange(5).cuda(), frequencies(32).cuda(), *w, 1e-6 if norm else None)
    used = out if read == "both" else [out["qk".index(read)]]
    leaves = [q, k] + [t for t in w if norm]
    got = torch.autograd.grad(used, leaves, [torch.ones_like(t) for t in used], allow_unused=True)
    for n, (x, d) in enumerate(zip((q, k), got)):
        if read in ("both", "qk"[n]):
            assert d.shape == x.shape and d.dtype == x.dtype and (d.numel() == 0 or d.any())
        if norm:
            met = x.shape[1] > 0 and read in ("both", "qk"[n])
            assert got[2 + n].shape == (64,) and bool(got[2 + n].any()) == met


def test_gradients_where_neither_output_counts():
    """Zeros for the weights where what reads the outputs hands no gradient back."""
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope

    class Drop(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k):
            return q.sum() + k.sum()

        @staticmethod
        def backward(ctx, d):
            return None, None
    q, k = (rand((5, n, 64), torch.float32, n).cuda().requires_grad_(True) for n in (4, 2))
    w = torch.ones(64, device="cuda", requires_grad=True)
    out = qk_norm_rope(q, k, torch.arange(5).cuda(), frequencies(32).cuda(), w, w, 1e-6)
    Drop.apply(*out).backward()
    assert q.grad is None and k.grad is None and (w.grad is None or not w.grad.any())


def test_the_c_named_call():
    import mxfp4_quantized_gemm_amd as mx
    none, pos, freq = torch.empty(5, 0, 64, device="cuda"), torch.arange(5).cuda(), frequencies(32).cuda()
    w, dw = torch.ones(64, device="cuda"), torch.full((2, 64), 7.0, device="cuda")
    ws = torch.empty(mx.mxfp4_qk_norm_rope_bwd_workspace_bytes(5, 0, 0, 64), dtype=torch.uint8, device="cuda")
    rstd = torch.empty(5, 0, device="cuda")
    mx.mxfp4_qk_norm_rope(none, none, pos, freq, w, w, 1e-6, none, none, rstd)
    mx.mxfp4_qk_norm_rope_bwd(none, none, none, none, pos, freq, w, w, rstd, none, none, dw[0], dw[1], ws)
    assert not dw.any()
