"""The C-named calls of attention's operators refuse operands on different GPUs, whose
addresses a kernel on one of them must not be given. (Stand-ins for tensors of two GPUs;
nothing is launched.)"""
import pytest
import torch

import mxfp4_quantized_gemm_amd as mx

BF16, F32, F64, I8, I32, I64, U8 = (torch.bfloat16, torch.float32, torch.float64, torch.int8, torch.int32, torch.int64,
                                    torch.uint8)


class Stand:
    """A contiguous tensor on GPU 0 that has everything but memory."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def size(self, i):
        return self.shape[i]

    def stride(self, i=None):
        s = [self.shape[j + 1:].numel() for j in range(len(self.shape))]
        return tuple(s) if i is None else s[i]

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


def calls():
    """Arguments by name; those of the cache as cache_0 to cache_3."""
    q = lambda: Stand(BF16, 5, 4, 64)
    k = lambda: Stand(BF16, 5, 2, 64)
    w = lambda: Stand(BF16, 64)
    turn = lambda: dict(positions=Stand(I64, 5), frequencies=Stand(F64, 32), q_weight=w(), k_weight=w())
    cache = lambda: dict(cache_0=Stand(I8, 8, 2, 16, 64), cache_1=Stand(F32, 8, 2, 16), cache_2=Stand(I8, 8, 2, 16, 64),
                         cache_3=Stand(F32, 8, 2, 16))
    return {
        "mxfp4_qk_norm_rope": dict(q=q(), k=k(), **turn(), eps=1e-6, q_out=q(), k_out=k(), rstd=Stand(F32, 5, 6)),
        "mxfp4_qk_norm_rope_bwd": dict(dq=q(), dk=k(), q=q(), k=k(), **turn(), rstd=Stand(F32, 5, 6), dq_out=q(),
                                       dk_out=k(), dq_weight=w(), dk_weight=w(), ws=Stand(U8, 1 << 20)),
        "mxfp4_int8_kv_write": dict(q=q(), k=k(), v=k(), **turn(), eps=1e-6, **cache(), slots=Stand(I64, 5), q_out=q()),
        "mxfp4_int8_kv_read": dict(**cache(), slots=Stand(I64, 5), k=k(), v=k()),
        "mxfp4_paged_attention": dict(q=q(), **cache(), pages=Stand(I32, 5, 3), lengths=Stand(I32, 5), scale=0.125,
                                      window=0, out=q(), lse=Stand(F32, 5, 4), ws=Stand(U8, 1 << 20)),
    }


def call(name, args):
    cache = [args.pop(f"cache_{i}") for i in range(4) if f"cache_{i}" in args]
    getattr(mx, name)(**args, **({"cache": cache} if cache else {}))


@pytest.mark.parametrize("name", list(calls()))
def test_operands_on_different_gpus_are_refused(name, monkeypatch):
    launched = []
    monkeypatch.setattr(mx, "_run", lambda fn, *a: launched.append(fn.__name__))
    call(name, calls()[name])
    assert launched == [name]
    for k, t in calls()[name].items():
        if isinstance(t, Stand):
            args = calls()[name]
            args[k].device = torch.device("cuda", 1)
            with pytest.raises(ValueError, match="must be on"):
                call(name, args)
            assert launched == [name], k
