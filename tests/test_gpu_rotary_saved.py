"""What qk_norm_rope keeps for its gradient: without a norm that is the turn back alone,
which reads neither queries nor keys."""
import pytest
import torch

from tests.attention_util import frequencies, rand

pytestmark = pytest.mark.gpu


def inputs(T=7, H=4, K=2, D=64, dtype=torch.bfloat16):
    q, k = (rand((T, n, D), dtype, n).cuda().requires_grad_(True) for n in (H, K))
    return q, k, torch.arange(T).cuda() * 5 + 3, frequencies(D // 2).cuda()


def test_without_a_norm_the_heads_may_change():
    """The same gradients whether queries and keys are overwritten after the call or not."""
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope
    q, k, pos, freq = inputs()
    dq, dk = rand(q.shape, q.dtype, 8).cuda(), rand(k.shape, k.dtype, 9).cuda()
    want = torch.autograd.grad(qk_norm_rope(q, k, pos, freq), (q, k), (dq, dk))
    q1, k1 = q * 1, k * 1
    out = qk_norm_rope(q1, k1, pos, freq)
    with torch.no_grad():
        q1.fill_(float("nan"))
        k1.mul_(2)
    got = torch.autograd.grad(out, (q, k), (dq, dk))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # one output alone, leading dimensions, and heads that are views of a product's rows
    rows = rand((2, 3, 6, 64), torch.float32, 10).cuda().requires_grad_(True)
    out = qk_norm_rope(*rows.split([4, 2], 2), pos[:6].view(2, 3), freq)
    g, = torch.autograd.grad(out[1], rows, torch.ones_like(out[1]), retain_graph=True)
    both, = torch.autograd.grad(out, rows, [torch.ones_like(t) for t in out])
    assert torch.equal(g[:, :, 4:], both[:, :, 4:]) and not g[:, :, :4].any() and both[:, :, :4].any()


def test_without_a_norm_the_heads_are_not_kept():
    """Their memory is free again once the caller drops them."""
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope
    q, k, pos, freq = inputs(T=4096, H=8, K=8)
    size = q.numel() * 2 + k.numel() * 2
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    q1, k1 = q * 1, k * 1
    out = qk_norm_rope(q1, k1, pos, freq)
    del q1, k1
    kept = torch.cuda.memory_allocated() - before - size  # but for the outputs
    assert kept < size // 8, kept
    del out


def test_with_a_norm_a_change_of_the_heads_is_seen():
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope
    for which in (0, 1):
        q, k, pos, freq = inputs()
        x = [q * 1, k * 1]
        out = qk_norm_rope(*x, pos, freq, eps=1e-6)
        with torch.no_grad():
            x[which].mul_(2)
        with pytest.raises(RuntimeError, match="inplace"):
            torch.autograd.grad(out, (q, k), [torch.ones_like(t) for t in out])


def test_positions_and_frequencies_that_change_are_seen():
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope
    for which in (2, 3):
        a = inputs()
        out = qk_norm_rope(*a)
        a[which].add_(1)
        with pytest.raises(RuntimeError, match="inplace"):
            torch.autograd.grad(out, a[:2], [torch.ones_like(t) for t in out])
