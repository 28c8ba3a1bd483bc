"""A feed-forward block trained in MXFP4 and served in 8 bits.

    python examples/feed_forward_int8.py [--hidden 1024] [--inner 3584] [--steps 20]

Trains norm -> gate and up (MXFP4Linear) -> silu(gate) * up -> down (MXFP4Linear)
with the residual stream on a synthetic target for a few steps (RMSNorm's
gradient feeds the norm's weight and the stream), then quantizes the trained
weights to int8 codes with a scale a channel and runs the same block on a
prompt and on single tokens with int8_mlp, and says how far the 8-bit block is
from the trained weights in 32 bits.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mxfp4_quantized_gemm_amd.int8 import int8_mlp, int8_quantize  # noqa: E402
from mxfp4_quantized_gemm_amd.linear import MXFP4Linear  # noqa: E402
from mxfp4_quantized_gemm_amd.norm import RMSNorm  # noqa: E402


class FeedForward(torch.nn.Module):
    def __init__(self, hidden, inner, device):
        super().__init__()
        self.inner = inner
        self.norm = RMSNorm(hidden, device=device)
        self.gate_up = MXFP4Linear(hidden, 2 * inner, device=device)
        self.down = MXFP4Linear(inner, hidden, device=device)

    def forward(self, x, residual):
        y, h = self.norm(x, residual)
        gu = self.gate_up(y)
        return self.down(torch.nn.functional.silu(gu[..., :self.inner]) * gu[..., self.inner:]), h

    @torch.no_grad()
    def reference(self, x, residual):
        """The block with the trained weights in 32 bits."""
        h = (x.float() + residual.float()).to(x.dtype).float()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + self.norm.eps) * self.norm.weight.float()
        gu = y @ self.gate_up.weight.float().t()
        return (torch.nn.functional.silu(gu[..., :self.inner]) * gu[..., self.inner:]) @ self.down.weight.float().t()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=3584)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    block = FeedForward(a.hidden, a.inner, "cuda")
    x, res = (torch.randn(a.tokens, a.hidden, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    target = torch.randn(a.tokens, a.hidden, device="cuda")
    opt = torch.optim.SGD(block.parameters(), lr=20.0)
    losses = []
    for _ in range(a.steps):
        y, h = block(x, res)
        loss = (y.float() + h.float() - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    print(f"training loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")

    with torch.no_grad():
        gu, gus = int8_quantize(block.gate_up.weight)
        dn, dns = int8_quantize(block.down.weight)
        want = block.reference(x, res)
        far = {}
        for name, n in (("prompt", a.tokens), ("one token", 1)):
            y, h = int8_mlp(x[:n], block.norm.weight, block.norm.eps, gu, gus, dn, dns, residual=res[:n])
            far[name] = float((y.float() - want[:n]).norm() / want[:n].norm())
            print(f"8-bit block, {name}: {far[name]:.4f} from the weights in 32 bits")
    return losses, far


if __name__ == "__main__":
    main()
