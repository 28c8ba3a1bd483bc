"""The cache read back in more rows than a launch takes."""
import pytest
import torch

from tests.attention_util import make_cache

pytestmark = pytest.mark.gpu


def test_more_rows_than_a_launch_takes():
    """2^27 rows of codes are a launch, 65536 tokens of 1024 heads: on both sides of its end, and at the
    beginning, the values as in a call of their own."""
    from mxfp4_quantized_gemm_amd.kv_cache import int8_kv_read
    T = 65536 + 5
    cache = [t.cuda() for t in make_cache(2, 1024, 16, 1, 1)]
    slots = torch.randint(-2, 34, (T,), generator=torch.Generator().manual_seed(2)).cuda()
    whole = int8_kv_read(cache, slots, 1)
    for at in (slice(0, 7), slice(65536 - 7, T), slice(65536, T)):
        for a, b in zip(whole, int8_kv_read(cache, slots[at].contiguous(), 1)):
            assert a.shape == (T, 1024, 1) and torch.equal(a[at], b) and b.any()
