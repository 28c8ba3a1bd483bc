"""Infinite scales of tokens that count, and scores of -infinity."""
import pytest
import torch

from tests.attention_util import TYPES, U, attend64, half_step, make_cache, near

pytestmark = pytest.mark.gpu
INF, D = float("inf"), 64


def attend(cache, n, q):
    from mxfp4_quantized_gemm_amd.attention import paged_attention
    return paged_attention(q.cuda(), [t.cuda() for t in cache], torch.arange(cache[0].shape[0], dtype=torch.int32)[None].cuda(),
                           torch.tensor([n], dtype=torch.int32).cuda(), return_lse=True)


def without(cache, n, at):
    """The cache of the first n tokens but the one at `at`, side by side."""
    keep = torch.arange(n)[torch.arange(n) != at]
    out = []
    for t in cache:
        rows = t[keep // 16, :, keep % 16]  # [tokens][heads]...
        to = torch.zeros(-(-max(n - 1, 1) // 16) * 16, *rows.shape[1:], dtype=t.dtype)
        to[: n - 1] = rows
        out.append(to.reshape(-1, 16, *rows.shape[1:]).transpose(1, 2).contiguous())
    return out


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,at", [(9, 3), (9, 0), (700, 600), (5000, 4999)])
def test_an_infinite_key_scale(n, at, dtype):
    """The token's score is an infinity of the product's sign, NaN where the product is 0. One of -infinity
    is a probability of 0; one of +infinity leaves no number."""
    cache, dt = make_cache(-(-n // 16), 1, 16, D, n), TYPES[dtype]
    q = torch.ones(1, 2, D, dtype=dt)
    rest = without(cache, n, at)
    o, lse, tol = attend64(q, rest, torch.arange(rest[0].shape[0], dtype=torch.int32)[None], [n - 1], D ** -0.5, 0, dt, 2 * U)
    # a score's error as attend64 has it, and the sum's of n tokens
    size = float((rest[0].double().abs().sum(-1) * rest[1].double()).max()) * D ** -0.5
    lse_tol = ((D + 16) * U * size + 2 * (n + 64) * U) * torch.ones_like(lse) + 8 * U * lse.abs()
    for scale in (INF, -INF):
        for code in (1, -1, 0):
            cache[0][at // 16, 0, at % 16], cache[1][at // 16, 0, at % 16] = code, scale
            got, got_lse = attend(cache, n, q)
            if scale * code == -INF:
                near(got, o, tol + half_step(o, dt), "o")
                near(got_lse, lse, lse_tol, "lse")
            else:
                assert got.isnan().all() and got_lse.isnan().all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,at", [(9, 3), (700, 600), (5000, 4999)])
def test_an_infinite_value_scale(n, at, dtype):
    """No number in any column, as of a NaN, whether the token's probability is 0 or not."""
    cache = make_cache(-(-n // 16), 1, 16, D, n)
    cache[1].fill_(2.0 ** -12)  # scores of at most 2
    for k_scale in (2.0 ** -12, -INF):
        cache[0][at // 16, 0, at % 16], cache[1][at // 16, 0, at % 16] = 1, k_scale
        for scale in (INF, -INF, float("nan")):
            cache[3][at // 16, 0, at % 16] = scale
            o, lse = attend(cache, n, torch.ones(1, 2, D, dtype=TYPES[dtype]))
            assert o.isnan().all() and lse.isfinite().all()


@pytest.mark.parametrize("n", [1, 50, 700, 5000])
def test_scores_of_minus_infinity_alone(n):
    """No token has a probability: zeros, as for a sequence without one, however it is cut."""
    cache = make_cache(-(-n // 16), 1, 16, D, n)
    cache[0].fill_(1)
    cache[1].fill_(-INF)
    o, lse = attend(cache, n, torch.ones(1, 2, D, dtype=torch.bfloat16))
    assert not o.any() and (lse == -INF).all()
