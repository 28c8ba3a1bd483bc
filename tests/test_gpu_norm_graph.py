"""A training step's norm, forward and backward, recorded into a HIP graph:
every replay equals the eager result, with the inputs overwritten and other
work in between. (Gradients are taken with autograd.grad, and no eager graph of
the recorded leaves is alive meanwhile.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.mark.parametrize("rows,cols", [(40, 256), (600, 1111), (700, 4096)])
def test_gradient_replays(rows, cols):
    from mxfp4_quantized_gemm_amd.norm import rms_norm

    def rand(*shape, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.randn(*shape, device="cuda", generator=g).bfloat16()
    data = [rand(rows, cols, seed=0), rand(rows, cols, seed=1), rand(cols, seed=2) + 1]
    dy, dh = rand(rows, cols, seed=3), rand(rows, cols, seed=4)

    def step(leaves):
        y, h = rms_norm(leaves[0], leaves[2], EPS, residual=leaves[1])
        return (y.detach(), h.detach(), *torch.autograd.grad((y, h), leaves, (dy, dh)))

    def eager():  # on leaves of its own
        return step([t.detach().clone().requires_grad_(True) for t in data])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    leaves = [t.clone().requires_grad_(True) for t in data]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(leaves)
    for i in range(4):
        data[0].copy_(rand(rows, cols, seed=10 + i))
        dy.copy_(rand(rows, cols, seed=20 + i))
        want = eager()
        with torch.no_grad():
            leaves[0].copy_(data[0])
        torch.cuda.synchronize()
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        torch.randn(1000, device="cuda").sum()
