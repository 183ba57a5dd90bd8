"""Sparse attention by blocks of a paged cache, and the cache's pages between steps (``include/tks_blocks.h``).

Over the cache of ``attention.py``, as thin calls over ``libtks.so``:

    tks.cache_bounds(k_cache, page_table, lens, bounds, start=old, scales=scales)   # after a write
    scores, seen = tks.block_scores(q, bounds, page_table, kv_len, block, first=1, last=1)
    picked = tks.topk_indices(scores.flatten(0, 2), n, row_len=seen.flatten())      # the selector
    out = tks.block_attention(q, k_cache, v_cache, page_table, picked.view(*seen.shape, n), block,
                              kv_len=kv_len, scales=scales)

    table, src, dst = tks.cache_fork(page_table, lens, parents, lens + 1, pages, page_size)
    tks.cache_copy(src, dst, k_cache, v_cache, scales=scales, bounds=bounds)        # for every layer

A sequence's block j is its positions ``[j * block, (j + 1) * block)``.  A sequence of n tokens
holds the first ``ceil(n / page_size)`` pages of its page table's row; a page that no sequence
holds is free.
"""

from __future__ import annotations

import ctypes
import threading

from . import attention as _attention
from .attention import _I32, _I64, _VP, _handle

TKS_E_NO_PAGE = 9


class Bounds(ctypes.Structure):
    """``tks_bounds``: the bounds of a cache's blocks as the C ABI sees them."""

    _fields_ = [("bounds", _VP), ("block", _I32), ("pages", _I32), ("page_size", _I32), ("kv_heads", _I32), ("head_dim", _I32)]


SIGNATURES = {
    "tks_cache_bounds": (ctypes.c_int, [_VP, _VP, _VP, _I64, _I32, _I32, _VP, _VP, _VP]),
    "tks_block_scores": (ctypes.c_int, [_VP, _VP, _VP, _I32, _I32, _VP, _I32, _VP, _VP]),
    "tks_block_attention": (ctypes.c_int, [_VP, _VP, _VP, _I32, _I32, _VP, _VP]),
    "tks_cache_fork": (ctypes.c_int, [_VP, _I64, _I32, _I32, _VP, _VP, _VP, _I32, _VP, _I32, _I32, _VP, _VP, _VP, _VP, _VP]),
    "tks_cache_compact": (ctypes.c_int, [_VP, _I64, _I32, _I32, _VP, _VP, _I32, _I32, _VP, _VP, _VP, _VP, _VP, _VP]),
    "tks_cache_copy": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _VP, _VP]),
}

_pointed = (None, None)  # the C++ module and the library that its calls of this part go to
_change = threading.Lock()


def _native():
    """The C++ module, with the calls of this part going to the library in use."""
    global _pointed
    module = _attention._binding or _attention._native()
    library = _attention._library
    if _pointed[0] is not module or _pointed[1] is not library:
        from . import TksError

        with _change:
            module.set_blocks(TksError, *(ctypes.cast(getattr(library, name), _VP).value for name in SIGNATURES))
            _pointed = (module, library)
    return module


def cache_bounds(k_cache, page_table, end, bounds, start=None, scales=None, stream=None):
    """Brings the bounds of the blocks that positions ``[start[b], end[b])`` lie in up to date.

    ``bounds``: bfloat16 CUDA tensor [pages, page_size // block, kv_heads, 2, head_dim], the least
    and the largest value of each block's keys in every channel; only the blocks named are written.
    ``page_table``: int32 [batch, n]; ``end``: int32 [batch], the sequences' lengths; ``start``:
    int32 [batch], the lengths before the last write (None: 0).  A block of a page that several of the
    sequences hold, at one place of their rows, is taken up to the furthest of their ends.
    """
    _native().bounds(k_cache, page_table, end, bounds, start, scales, _handle(stream))


def block_scores(q, bounds, page_table, kv_len, block, first=0, last=0, n=None, out=None, stream=None):
    """How large a product the blocks' keys can have with each token's queries: what to select blocks by.

    ``q``: bfloat16 [batch, tokens, q_heads, head_dim]; ``bounds`` as ``cache_bounds`` keeps them;
    ``kv_len``: int32 [batch, tokens], the positions that a token sees (None: all).  The score of a
    block, for a token and key/value head, is the largest over the head's query heads of
    ``sum_d max(q_d * least_d, q_d * largest_d)``; a token's ``first`` first and ``last`` last blocks
    score +inf, blocks that it does not see -inf.  No (finite) key of a bfloat16 cache has a larger
    product than its block's score; of an int8 one, by at most 2^-8 of the terms' magnitudes, as the
    bounds are rounded to nearest.

    Returns (scores, seen): float32 [batch, tokens, kv_heads, n], of the row's first n blocks (None:
    all that the page table has room for), and int32 [batch, tokens, kv_heads], how many of them the
    token sees, which ``topk_indices`` takes as ``row_len``.
    """
    return _native().scores(q, bounds, page_table, kv_len, block, first, last, n, out, _handle(stream))


def block_attention(q, k_cache, v_cache, page_table, blocks, block, kv_len=None, scales=None, softmax_scale=None, out=None,
                    return_lse=False, stream=None):
    """Attention of each query token and key/value head over its own list of blocks.

    ``q`` and ``page_table`` as in ``tree_attention``.  ``blocks``: int32 [batch, tokens, kv_heads,
    n], in any order, negative entries are skipped; ``kv_len``: int32 [batch, tokens], the positions
    that a token sees (None: all of the page table).  A block that starts beyond them is skipped and
    reported by ``device_status``.  Returns as ``tree_attention`` does.
    """
    return _native().block(q, k_cache, v_cache, page_table, blocks, block, kv_len, scales, softmax_scale, out, bool(return_lse),
                           _handle(stream))


def cache_fork(page_table, lens, parents, new_lens, pages, page_size, keep=None, out=None, stream=None):
    """The page tables of the next step's sequences, each a continuation of one of this step's.

    ``page_table``: int32 [sequences, n] and ``lens``: int32 [sequences], as they are.  ``parents``:
    int32 [children], the sequence that a child goes on from (negative: none); ``new_lens``: int32
    [children], the length that it is to have pages for (shorter than its parent's: it is cut).  A
    sequence without a child has ended, and its pages are free.  ``keep``: bool or uint8 [pages],
    pages that something else holds.

    Returns (table, src, dst): int32 [children, n], -1 behind each child's pages, and int32
    [children] twice, the pages to copy (``cache_copy``, for every layer), or -1: a child that is
    going to write to a partly filled page that another child holds too gets a copy of it.  Free
    pages are taken lowest first; where none is left, entries are -1 and ``device_status`` says
    ``TKS_E_NO_PAGE``.
    """
    return _native().fork(page_table, lens, parents, new_lens, pages, page_size, keep, out, _handle(stream))


def cache_compact(page_table, lens, pages, page_size, keep=None, out=None, stream=None):
    """Moves the pages in use to the lowest ones (those of ``keep`` stay where they are).

    Returns (table, src, dst, count): the page table afterwards (``out``: it may be the old one
    itself), the moves for ``cache_copy``, int32 [pages // 2] each with -1 behind the last, and int32
    [2]: the number of moves, and of pages in use.
    """
    return _native().compact(page_table, lens, pages, page_size, keep, out, _handle(stream))


def cache_copy(src, dst, k_cache, v_cache, scales=None, bounds=None, count=None, stream=None):
    """Copies pages ``src[i]`` to ``dst[i]`` of a cache: keys, values, scales and, where given, bounds.

    ``src``, ``dst``: int32 [n]; pairs with a negative page are skipped.  ``count``: an int32 CUDA
    tensor whose first element says how many pairs there are (as ``cache_compact`` returns it).
    No page may be in ``dst`` twice, or in both.
    """
    _native().copy(src, dst, k_cache, v_cache, scales, bounds, count, _handle(stream))
