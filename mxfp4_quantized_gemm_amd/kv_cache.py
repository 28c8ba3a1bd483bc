"""A cache of keys and values in 8 bits, in pages: int8 codes with one scale for
each token and head, as ``int8_quantize`` makes them of a row.

    cache = int8_kv_cache(pages, kv_heads, head_dim)      zeros
    int8_kv_write(k, v, cache, slots)                     codes of k and v
    q = int8_kv_append(q, k, v, cache, slots, ...)        norm, rotation and codes in one pass
    k, v = int8_kv_read(cache, slots, head_dim)           what the codes stand for

A slot is a token's place, page * page_size + row. A token whose slot is
negative or past the cache is not written, and reads as zeros; of tokens with the
same slot in one call the last one stays. ``paged_attention`` in attention.py
reads the cache. Inference only: inputs that require a gradient are refused.
Marshalling only: every step runs in the library's kernels.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._load import ops


class Int8KVCache(NamedTuple):
    """Codes [pages][heads][page size][pitch], the pitch being the width of a head
    rounded up to a multiple of 64, and float32 scales [pages][heads][page size].
    The functions here take any four such tensors in this order."""
    k: torch.Tensor
    k_scales: torch.Tensor
    v: torch.Tensor
    v_scales: torch.Tensor


def int8_kv_cache(pages, kv_heads, head_dim, page_size=64, device="cuda"):
    """An empty cache; page_size is a multiple of 16, pages * page_size below 2^31."""
    if page_size < 16 or page_size % 16:
        raise ValueError(f"page_size must be a multiple of 16, got {page_size}")
    if not 1 <= head_dim <= 256:
        raise ValueError(f"head_dim must be from 1 to 256, got {head_dim}")
    shape = (pages, kv_heads, page_size)
    codes = lambda: torch.zeros(*shape, (head_dim + 63) // 64 * 64, dtype=torch.int8, device=device)  # noqa: E731
    scales = lambda: torch.zeros(shape, dtype=torch.float32, device=device)  # noqa: E731
    return Int8KVCache(codes(), scales(), codes(), scales())


def int8_kv_write(k, v, cache, slots):
    """Codes of k and v [..., kv heads, head_dim] into the cache at slots [...] (int64)."""
    ops.int8_kv_write(k, v, *cache, slots)


def int8_kv_append(q, k, v, cache, slots, positions, frequencies, q_weight=None, k_weight=None, eps=None,
                   sections=None, interleaved=False):
    """``qk_norm_rope`` of q and k with k's result and v written to the cache
    (from 32 bits, without a rounding in between); returns q'."""
    return ops.int8_kv_append(q, k, v, *cache, slots, positions, frequencies, q_weight, k_weight, eps, sections,
                              interleaved)


def int8_kv_read(cache, slots, head_dim, dtype=torch.bfloat16):
    """(k, v) [..., kv heads, head_dim] of the tokens at slots [...], code times scale."""
    return ops.int8_kv_read(*cache, slots, head_dim, dtype)
