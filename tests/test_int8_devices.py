"""The C-named norm and 8-bit calls refuse operands on different GPUs, whose
addresses a kernel on one of them must not be given. (Stand-ins for tensors of
two GPUs; nothing is launched.)"""
import pytest
import torch

import mxfp4_quantized_gemm_amd as mx

BF16, F32, I8, U8 = torch.bfloat16, torch.float32, torch.int8, torch.uint8


class Stand:
    """A contiguous tensor on GPU 0 that has everything but memory."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def size(self, i):
        return self.shape[i]

    def stride(self):
        return (self.shape[1], 1) if self.dim() == 2 else (1,)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


def calls():
    m = lambda dtype=BF16: Stand(dtype, 4, 128)
    v = lambda dtype=F32, n=128: Stand(dtype, n)
    return {
        "mxfp4_rmsnorm": dict(x=m(), residual=m(), weight=v(BF16), eps=1e-5, h=m(), y=m(), rstd=v(n=4)),
        "mxfp4_rmsnorm_int8": dict(x=m(), residual=m(), weight=v(), eps=1e-5, h=m(), codes=m(I8), scales=v(n=4)),
        "mxfp4_rmsnorm_bwd": dict(dy=m(), dh=m(), h=m(), weight=v(), rstd=v(n=4), dx=m(), dweight=v(), ws=v(U8, 1 << 20)),
        "mxfp4_int8_quantize": dict(x=m(), gate=m(), codes=m(I8), scales=v(n=4)),
        "mxfp4_int8_gemm": dict(A=m(I8), a_scales=v(n=4), B=Stand(I8, 8, 128), b_scales=v(n=8), bias=v(n=8),
                                C=Stand(BF16, 4, 8), ws=v(U8, 1 << 20)),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_operands_on_different_gpus_are_refused(name, monkeypatch):
    launched = []
    monkeypatch.setattr(mx, "_run", lambda fn, *a: launched.append(fn.__name__))
    getattr(mx, name)(**calls()[name])
    assert launched == [name]
    for k, t in calls()[name].items():
        if isinstance(t, Stand):
            args = calls()[name]
            args[k].device = torch.device("cuda", 1)
            with pytest.raises(ValueError, match="must be on"):
                getattr(mx, name)(**args)
            assert launched == [name], k
