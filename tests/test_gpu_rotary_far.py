"""Norm and rotation of far positions, and of more tokens than a launch takes."""
import pytest
import torch

from tests.attention_util import U, angles, frequencies, half_step, near, rand, turned

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inter", [False, True])
def test_positions_up_to_2_to_the_40(inter):
    """An angle is its fp64 product; quarter turns of it round twice more there (the factor 2 / pi
    and its product), 2^-52 of the angle, which counts where the angle is large."""
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope
    T, D = 60, 64
    pos = torch.randint(-(1 << 40), 1 << 40, (T,), generator=torch.Generator().manual_seed(1))
    pos[0], pos[1] = (1 << 40) - 1, -(1 << 40)
    q, k, freq = rand((T, 3, D), torch.float32, 2), rand((T, 1, D), torch.float32, 3), frequencies(D // 2)
    a = angles(pos, freq, None)
    assert float(a.abs().max()) > 2.0 ** 39
    out = qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), freq.cuda(), interleaved=inter)
    for x, got in zip((q, k), out):
        y, tol = turned(x, None, None, a, inter)
        wide = a.abs() * 2.0 ** -52
        wide = wide.repeat_interleave(2, 1) if inter else torch.cat([wide, wide], 1)
        near(got, y, tol + tol / (8 * U) * wide[:, None] + half_step(y, torch.float32), "turned")


def test_more_tokens_than_a_launch_takes():
    """2^22 tokens are a launch: the last of the first one and those of the next as in a call of their own."""
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope
    T, D, cut = (1 << 22) + 3, 4, (1 << 22) - 6
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q, k, dq, dk = (torch.randn(T, 1, D, device="cuda", generator=g).bfloat16() for _ in range(4))
    pos, freq = torch.randint(0, 5000, (2, T), device="cuda", generator=g), frequencies(2).cuda()
    w = [(1 + 0.1 * rand((D,), torch.float32, i)).cuda() for i in (2, 3)]

    def call(at):
        x = [q[at].detach().requires_grad_(True), k[at].detach().requires_grad_(True)]
        out = qk_norm_rope(*x, pos[:, at].contiguous(), freq, *w, 1e-6, sections=(1, 1))
        return (*out, *torch.autograd.grad(out, x, (dq[at], dk[at])))
    whole, end = call(slice(0, T)), call(slice(cut, T))
    begin = call(slice(0, 9))
    for a, b, c in zip(whole, end, begin):
        assert torch.equal(a[cut:], b) and torch.equal(a[:9], c) and a[cut:].isfinite().all()
    assert whole[0][cut:].any(-1).all() and whole[2][cut:].any(-1).all()
