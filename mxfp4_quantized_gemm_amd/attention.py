"""Attention of one new token a sequence over an int8 cache of keys and values
in pages (kv_cache.py), and the attention block in 8 bits.

    o = paged_attention(q, cache, pages, lengths)     softmax(scale q k^T) v
    y, h = int8_attention(x, ...)                     norm to output product

The lengths and page tables stay on the GPU, so a captured graph serves sequences
as they grow. The work is cut by the tables' width, which the host knows: one or two
sequences take two to six times as long by a table for 131072 tokens as by one of their
own length up to 8192, and graphs for a few widths serve them better than one.
Inference only: inputs that require a gradient are refused.
Marshalling only: every step runs in the library's kernels.
"""
from __future__ import annotations

from ._load import ops


def paged_attention(q, cache, pages, lengths, scale=None, window=0, return_lse=False):
    """q [batch][heads][dim] -> [batch][heads][dim] in its type; the heads are a
    multiple of the cache's, of which each serves as many neighbouring ones.

    Sequence b attends to its first lengths[b] tokens (int32), the last ``window``
    of them if window > 0; token t is row t % page_size of page
    pages[b][t // page_size] (int32). A sequence without tokens gives zeros;
    tokens of a page that is not in the cache (-1, say) do not count. A score of
    -infinity (of an infinite query or key scale) is a probability of 0, and a sequence
    with no other gives zeros; one of +infinity or NaN gives NaN.
    scale: dim^-1/2 if None. return_lse: also the logarithm of the sum of the
    scores' exponentials, float32 [batch][heads].
    """
    return ops.paged_attention(q, *cache, pages, lengths, scale, window, return_lse)


def int8_attention(x, norm_weight, eps, qkv, qkv_scales, out, out_scales, cache, slots, pages, lengths, positions,
                   frequencies, q_weight=None, k_weight=None, qk_eps=None, *, head_dim, scale=None, window=0,
                   sections=None, interleaved=False, residual=None):
    """The attention block in 8 bits for one new token a sequence, as ``int8_mlp``
    is the feed-forward block: norm (of x + residual), query, key and value rows
    in one product (qkv: the query heads' rows first, then the key heads', then
    the value heads'; its result is held in x's type), norm and rotation of the
    heads with keys and values written to the cache at ``slots``, attention over
    ``lengths`` tokens (the new one among them), output product. Returns (y, h),
    h = x + residual (x itself without a residual)."""
    return ops.int8_attention(x, norm_weight, eps, qkv, qkv_scales, out, out_scales, *cache, slots, pages, lengths,
                              positions, frequencies, q_weight, k_weight, qk_eps, head_dim, scale, window, sections,
                              interleaved, residual)
