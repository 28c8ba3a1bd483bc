"""Norm of each head of queries and keys, and their rotation by position.

    u = x / sqrt(mean(x^2) + eps) * weight,  pairs (u_i, u_j) turned by position * frequency

``qk_norm_rope`` does both in one pass, with gradients (behind the
query-key-value product of an MXFP4Linear in training); ``int8_kv_append`` in
kv_cache.py is its form for serving. Marshalling only: every step runs in the
library's kernels.
"""
from __future__ import annotations

from ._load import ops


def qk_norm_rope(q, k, positions, frequencies, q_weight=None, k_weight=None, eps=None, sections=None,
                 interleaved=False):
    """(q', k'), of the inputs' type; differentiable once in q, k and the
    weights, in reverse mode (forward-mode tangents are refused). Without a norm the
    gradient needs neither q nor k: they are not kept for it, and may be overwritten.

    q [..., heads, dim] and k [..., key heads, dim], float32, bfloat16 or
    float16, any strides, dim up to 256. eps None: no norm, then no weights;
    weights [dim] of the heads' type or float32. frequencies float64 [pairs], in
    radians a position, 2 pairs <= dim (an empty one: no rotation): pair p is
    (p, pairs + p), or (2 p, 2 p + 1) if interleaved. positions int64 [...],
    or with sections (pairs of each of up to four axes, as time, height and
    width) [axes, ...].

    To capture a backward pass in a graph, keep no eager autograd graph of the same
    leaves alive, as for any operator under torch: it would put the leaves'
    accumulation on a stream that is not captured.
    """
    return ops.qk_norm_rope(q, k, positions, frequencies, q_weight, k_weight, eps, sections, interleaved)
