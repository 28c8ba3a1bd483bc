"""An eps that fp32 does not hold is refused by the norms of heads."""
import pytest
import torch

from tests.attention_util import frequencies, rand

pytestmark = pytest.mark.gpu


def test_eps_outside_32_bits_is_refused():
    """It is held in fp32: an eps that is infinite there would make every result 0, one that is 0 there
    would make a row of zeros NaN."""
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_append, int8_kv_cache
    from mxfp4_quantized_gemm_amd.rotary import qk_norm_rope
    x, pos, freq = rand((2, 1, 64), torch.float32, 1).cuda(), torch.arange(2).cuda(), frequencies(32).cuda()
    cache = int8_kv_cache(1, 1, 64, 16)
    before = [t.clone() for t in cache]
    for eps in (1e39, 1e300, 1e-46, 5e-324, float("inf"), float("nan"), -1e-6):
        with pytest.raises(ValueError, match="eps"):
            qk_norm_rope(x, x, pos, freq, eps=eps)
        with pytest.raises(ValueError, match="eps"):
            int8_kv_append(x, x, x, cache, pos, pos, freq, eps=eps)
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    zeros = torch.zeros(1, 1, 64, device="cuda")
    for eps in (3e38, 1.5e-45):  # the ends of what fp32 holds
        assert not qk_norm_rope(zeros, zeros, pos[:1], freq, eps=eps)[0].any()
    qk_norm_rope(x, x, pos, freq, eps=0.0)
