"""The paged key/value cache and the attention that reads it (``include/tks_attention.h``).

What stands around the selector in a decode step, as thin calls over ``libtks.so`` (tensors
are checked, and outputs allocated, by a small C++ module, ``csrc/tks_binding.cpp``):

    tks.cache_write(k, v, k_cache, v_cache, slots, scales=scales)      # the new tokens
    idx = tks.topk_indices(logits, 2048, row_len=lens)                 # the selector
    out = tks.selected_attention(q, k_cache, v_cache, pages, idx, scales=scales)
    out = tks.tree_attention(q, k_cache, v_cache, pages, ctx_len, tree=bits, scales=scales)

A cache is two CUDA tensors ``[pages, page_size, kv_heads, head_dim]``, bfloat16, or
int8 with ``scales``, float32 ``[pages, page_size, kv_heads, 2]`` (of the key and of the
value); slot ``s`` is token ``s % page_size`` of page ``s // page_size``.
"""

from __future__ import annotations

import ctypes
import threading

_I32, _I64, _VP, _F32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float

TKS_I8 = 2
TKS_E_INDEX = 8
TKS_DRAFTS_MAX = 1024


class Cache(ctypes.Structure):
    """``tks_cache``: a paged cache as the C ABI sees it (strides in elements)."""

    _fields_ = [("k", _VP), ("v", _VP), ("scales", _VP), ("held", _I32), ("pages", _I32),
                ("page_size", _I32), ("kv_heads", _I32), ("head_dim", _I32),
                ("page_stride", _I64), ("token_stride", _I64), ("head_stride", _I64)]


class Queries(ctypes.Structure):
    """``tks_queries``: the queries of an attention call as the C ABI sees them."""

    _fields_ = [("q", _VP), ("q_batch_stride", _I64), ("q_token_stride", _I64), ("q_head_stride", _I64),
                ("out", _VP), ("lse", _VP), ("batch", _I32), ("tokens", _I32), ("q_heads", _I32),
                ("page_table", _VP), ("table_stride", _I64), ("table_pages", _I32), ("softmax_scale", _F32)]


SIGNATURES = {
    "tks_cache_write": (ctypes.c_int, [_VP, _VP, _VP, _I32, _I32, _I64, _I64, _I64, _I64, _VP, _VP]),
    "tks_cache_read": (ctypes.c_int, [_VP, _VP, _I32, _VP, _VP, _I32, _VP]),
    "tks_tree_attention": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP]),
    "tks_selected_attention": (ctypes.c_int, [_VP, _VP, _VP, _I32, _VP, _VP]),
}


_binding = None  # the C++ module, once its calls have somewhere to go
_library = None  # the library that the package's calls go to
_first_use, _change = threading.Lock(), threading.Lock()


def _point(module):
    from . import TksError

    module.set_library(TksError, *(ctypes.cast(getattr(_library, name), _VP).value for name in SIGNATURES))


def bound(lib):
    """Makes the calls go to the entry points of `lib` (called when the package loads a library)."""
    global _library
    with _change:
        _library = lib
        if _binding is not None:
            _point(_binding)


def _native():
    """The C++ module that checks the tensors and makes the calls, built and loaded on first use."""
    global _binding
    with _first_use:
        if _binding is None:
            import importlib.util

            import torch  # noqa: F401  (its libraries come first)

            from . import load
            from ._build import build_binding

            spec = importlib.util.spec_from_file_location("tks_binding", build_binding())
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            load()
            with _change:
                _point(module)
                _binding = module  # (other threads' calls take it from here on)
    return _binding


def _handle(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def cache_write(k, v, k_cache, v_cache, slots, scales=None, stream=None):
    """Puts the keys and values of n tokens into a paged cache.

    ``k``, ``v``: bfloat16 or float32 CUDA tensors [n, kv_heads, head_dim] (views of a fused
    projection are read in place).  ``slots``: int32 CUDA tensor [n], where each goes, all
    different (what two tokens with one slot leave there is undefined); a negative slot skips
    its token.  An int8 cache takes each row as codes with a scale of
    max|x| / 127, written to ``scales``; a bfloat16 cache takes the values rounded.
    """
    (_binding or _native()).write(k, v, k_cache, v_cache, slots, scales, _handle(stream))


def cache_read(k_cache, v_cache, slots, scales=None, dtype=None, out=None, stream=None):
    """The keys and values that ``slots`` (int32 CUDA tensor [n]) stand for.

    Returns (k, v), ``dtype`` (bfloat16, the default, or float32) [n, kv_heads, head_dim];
    ``out``: a pair of contiguous CUDA tensors to fill.  Negative slots give zeros.
    """
    import torch

    if out is not None:
        dtype = out[0].dtype if dtype is None else dtype
    if dtype is not None and dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"dtype must be bfloat16 or float32, not {dtype}")
    k_out, v_out = (None, None) if out is None else out
    return (_binding or _native()).read(k_cache, v_cache, slots, scales, dtype is torch.float32, k_out, v_out, _handle(stream))


def tree_attention(q, k_cache, v_cache, page_table, ctx_len, tree=None, draft_len=None, scales=None,
                   softmax_scale=None, out=None, return_lse=False, stream=None):
    """Attention of drafted tokens over a cached context and over each other.

    ``q``: bfloat16 [batch, tokens, q_heads, head_dim]; query head h reads key/value head
    ``h // (q_heads // kv_heads)``.  ``page_table``: int32 [batch, n], position p of
    sequence b is in page ``page_table[b, p // page_size]``.  ``ctx_len``: int32 [batch],
    every query attends to the positions before it; the drafted tokens' own keys and values
    stand behind them, draft j at position ``ctx_len[b] + j``.  ``tree``: int32 [batch,
    tokens, ceil(tokens / 32)], query i attends to draft j where bit j % 32 of word j // 32
    is set (``tree_mask`` makes it from parents; None: a chain).  ``draft_len``: int32
    [batch], how many drafts a sequence has.  One token is an ordinary decode step.

    Returns bfloat16 like q, and with ``return_lse`` also float32 [batch, tokens, q_heads],
    the log-sum-exp of the attended, scaled scores.  A query that attends to nothing (one
    beyond ``draft_len`` too) gives zeros and -inf.
    """
    return (_binding or _native()).tree(q, k_cache, v_cache, page_table, ctx_len, tree, draft_len, scales, softmax_scale, out,
                                        bool(return_lse), _handle(stream))


def selected_attention(q, k_cache, v_cache, page_table, indices, kv_len=None, scales=None,
                       softmax_scale=None, out=None, return_lse=False, stream=None):
    """Attention of each query token over its own list of positions (what ``topk_indices`` returns).

    ``q`` and ``page_table`` as in ``tree_attention``.  ``indices``: int32 [batch, tokens, k]
    positions of sequence b, in any order, shared by the token's heads; negative entries are
    skipped, entries at or beyond ``kv_len[b]`` (int32 [batch], optional) are skipped and
    reported by ``device_status``.  Returns as ``tree_attention`` does.
    """
    return (_binding or _native()).selected(q, k_cache, v_cache, page_table, indices, kv_len, scales, softmax_scale, out,
                                            bool(return_lse), _handle(stream))


def tree_mask(parents):
    """The bits ``tree_attention`` takes, from each draft's parent.

    ``parents``: an integer tensor [batch, tokens]; the parent of draft i is an earlier draft
    of the same sequence, or -1 for one that follows the context directly.  A draft attends to
    itself, its parent, its parent's parent and so on.  Returns int32 [batch, tokens,
    ceil(tokens / 32)] on the parents' device.  The bits are made on the host (parents on a
    GPU are waited for), so keep them where the tree stays the same from step to step.
    """
    import torch

    rows = parents.tolist()
    words = (parents.shape[1] + 31) // 32
    table = []
    for row in rows:
        seen = []
        for i, p in enumerate(row):
            if not -1 <= p < i:
                raise ValueError(f"the parent of draft {i} must be -1 or an earlier draft, not {p}")
            seen.append((1 << i) | (seen[p] if p >= 0 else 0))
        table.append([[((m >> (32 * w)) & 0xFFFFFFFF) for w in range(words)] for m in seen])
    bits = torch.tensor(table, dtype=torch.int64).reshape(len(rows), parents.shape[1], words)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32).to(parents.device)
