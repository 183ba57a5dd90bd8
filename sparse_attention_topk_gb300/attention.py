"""The paged key/value cache and the attention that reads it (``include/tks_attention.h``).

What stands around the selector in a decode step, as thin calls over ``libtks.so``:

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


def _call(device, stream, fn):
    """fn(stream handle) with `device` current, and `stream` too (the device's current one if
    None), so that what fn allocates belongs to the stream that writes it."""
    import torch

    if stream is None and device.index == torch.cuda.current_device():
        return fn(torch.cuda.current_stream().cuda_stream)
    with torch.cuda.device(device):
        if stream is None:
            return fn(torch.cuda.current_stream().cuda_stream)
        s = stream
        if isinstance(stream, int):
            s = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream(device)
        with torch.cuda.stream(s):
            return fn(s.cuda_stream)


def _check(rc, what):
    if rc:
        from . import TksError
        raise TksError(rc, what)


def _cache(k_cache, v_cache, scales):
    import torch

    if k_cache.dim() != 4 or not k_cache.is_cuda:
        raise ValueError("caches must be CUDA tensors [pages, page_size, kv_heads, head_dim]")
    shape, stride, dtype = k_cache.shape, k_cache.stride(), k_cache.dtype
    if v_cache.shape != shape or v_cache.dtype != dtype or v_cache.stride() != stride or v_cache.device != k_cache.device:
        raise ValueError("k_cache and v_cache must have one shape, strides, dtype and device")
    pages, page_size, heads, dim = shape
    if dim not in (64, 128) or stride[3] != 1:
        raise ValueError("head_dim must be 64 or 128, and contiguous")
    if page_size < 1 or page_size & (page_size - 1):
        raise ValueError("page_size must be a power of two")
    if dtype is torch.int8:
        if scales is None or scales.shape != (pages, page_size, heads, 2) or scales.dtype is not torch.float32 \
                or not scales.is_contiguous() or scales.device != k_cache.device:
            raise ValueError("an int8 cache needs scales: a contiguous float32 CUDA tensor [pages, page_size, kv_heads, 2]")
        held, sc = TKS_I8, scales.data_ptr()
    elif dtype is torch.bfloat16:
        if scales is not None:
            raise ValueError("a bfloat16 cache has no scales")
        held, sc = 1, None
    else:
        raise ValueError(f"unsupported cache dtype {dtype}")
    return Cache(k_cache.data_ptr(), v_cache.data_ptr(), sc, held, pages, page_size, heads, dim, stride[0], stride[1], stride[2])


def _ints(t, shape, device, what):
    import torch

    if t.dtype is not torch.int32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 CUDA tensor {list(shape)} on the cache's device")
    return t.data_ptr()


def _rows_ok(t, size):
    """Whether the kernels can read t as it is: a contiguous last dimension, and 16-byte
    pieces everywhere else (an extent of one is never stepped over)."""
    unit = 16 // size
    return t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and \
        all(s >= 0 and s % unit == 0 for s, n in zip(t.stride()[:-1], t.shape[:-1]) if n > 1)


def _dtype(t, what):
    import torch

    if t is torch.bfloat16:
        return 1
    if t is torch.float32:
        return 0
    raise ValueError(f"{what} must be bfloat16 or float32, not {t}")


def cache_write(k, v, k_cache, v_cache, slots, scales=None, stream=None):
    """Puts the keys and values of n tokens into a paged cache.

    ``k``, ``v``: bfloat16 or float32 CUDA tensors [n, kv_heads, head_dim] (views of a fused
    projection are read in place).  ``slots``: int32 CUDA tensor [n], where each goes; a
    negative slot skips its token.  An int8 cache takes each row as codes with a scale of
    max|x| / 127, written to ``scales``; a bfloat16 cache takes the values rounded.
    """
    import torch

    c = _cache(k_cache, v_cache, scales)
    n, dev = slots.numel(), k_cache.device
    if k.shape != (n, c.kv_heads, c.head_dim) or v.shape != k.shape or v.dtype != k.dtype or k.device != dev or v.device != dev:
        raise ValueError(f"k and v must be CUDA tensors [{n}, {c.kv_heads}, {c.head_dim}] of one dtype on the cache's device")
    dt = _dtype(k.dtype, "k and v")
    at = _ints(slots, (n,), dev, "slots")
    if n == 0:
        return
    size = 4 if dt == 0 else 2

    def go(handle):
        a = k if _rows_ok(k, size) else k.contiguous()
        b = v if _rows_ok(v, size) else v.contiguous()
        if a.data_ptr() % 16 or b.data_ptr() % 16:
            a, b = a.clone(), b.clone()
        unit = 16 // size
        ks, vs = ([s if e > 1 else 0 for s, e in zip(t.stride(), t.shape)] for t in (a, b))
        return _lib().tks_cache_write(ctypes.byref(c), a.data_ptr(), b.data_ptr(), n, dt, ks[0], ks[1], vs[0], vs[1], at, handle)

    _check(_call(dev, stream, go), "tks_cache_write")


def cache_read(k_cache, v_cache, slots, scales=None, dtype=None, out=None, stream=None):
    """The keys and values that ``slots`` (int32 CUDA tensor [n]) stand for.

    Returns (k, v), ``dtype`` (bfloat16, the default, or float32) [n, kv_heads, head_dim];
    ``out``: a pair of contiguous CUDA tensors to fill.  Negative slots give zeros.
    """
    import torch

    c = _cache(k_cache, v_cache, scales)
    n, dev = slots.numel(), k_cache.device
    at = _ints(slots, (n,), dev, "slots")
    shape = (n, c.kv_heads, c.head_dim)
    if out is not None:
        dtype = out[0].dtype if dtype is None else dtype
        for t in out:
            if t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_contiguous() or t.data_ptr() % 16:
                raise ValueError(f"out must be two contiguous, 16-byte aligned {dtype} CUDA tensors {list(shape)}")
    dtype = torch.bfloat16 if dtype is None else dtype
    dt = _dtype(dtype, "dtype")
    result = []

    def go(handle):
        result.extend(out if out is not None else torch.empty((2,) + shape, dtype=dtype, device=dev))
        if n == 0:
            return 0
        return _lib().tks_cache_read(ctypes.byref(c), at, n, result[0].data_ptr(), result[1].data_ptr(), dt, handle)

    _check(_call(dev, stream, go), "tks_cache_read")
    return result[0], result[1]


def _attend(q, c, dev, page_table, softmax_scale, out, return_lse, stream, what, call):
    import torch

    if q.dim() != 4 or q.dtype is not torch.bfloat16 or q.device != dev or q.shape[3] != c.head_dim:
        raise ValueError(f"q must be a bfloat16 CUDA tensor [batch, tokens, q_heads, {c.head_dim}] on the cache's device")
    batch, tokens, heads, dim = q.shape
    if heads < 1 or heads % c.kv_heads:
        raise ValueError("q_heads must be a multiple of kv_heads")
    if page_table.dim() != 2 or page_table.shape[0] != batch or page_table.dtype is not torch.int32 \
            or page_table.device != dev or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be an int32 CUDA tensor [batch, pages of a sequence] with contiguous rows")
    if out is not None and (out.shape != q.shape or out.dtype is not torch.bfloat16 or out.device != dev
                            or not out.is_contiguous() or out.data_ptr() % 16):
        raise ValueError("out must be a contiguous, 16-byte aligned bfloat16 CUDA tensor of q's shape")
    scale = dim ** -0.5 if softmax_scale is None else float(softmax_scale)
    if not abs(scale) < float("inf"):
        raise ValueError("softmax_scale must be finite")
    result = []

    def go(handle):
        o = torch.empty(q.shape, dtype=q.dtype, device=dev) if out is None else out
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=dev) if return_lse else None
        result.extend((o, lse))
        x = q if _rows_ok(q, 2) else q.contiguous()
        if x.data_ptr() % 16:
            x = x.clone()
        st = [s if e > 1 else 0 for s, e in zip(x.stride(), x.shape)]
        queries = Queries(x.data_ptr(), st[0], st[1], st[2], o.data_ptr(), lse.data_ptr() if return_lse else None, batch, tokens, heads,
                          page_table.data_ptr(), page_table.stride(0) if batch > 1 else 0, page_table.shape[1], scale)
        return call(ctypes.byref(c), ctypes.byref(queries), handle)

    _check(_call(dev, stream, go), what)
    return tuple(result) if return_lse else result[0]


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
    c, dev = _cache(k_cache, v_cache, scales), k_cache.device
    batch, tokens = q.shape[0], q.shape[1]
    if tokens > TKS_DRAFTS_MAX:
        raise ValueError(f"at most {TKS_DRAFTS_MAX} drafted tokens")
    ctx = _ints(ctx_len, (batch,), dev, "ctx_len")
    count = None if draft_len is None else _ints(draft_len, (batch,), dev, "draft_len")
    bits = None if tree is None else _ints(tree, (batch, tokens, (tokens + 31) // 32), dev, "tree")
    return _attend(q, c, dev, page_table, softmax_scale, out, return_lse, stream, "tks_tree_attention",
                   lambda cache, queries, handle: _lib().tks_tree_attention(cache, queries, ctx, count, bits, handle))


def selected_attention(q, k_cache, v_cache, page_table, indices, kv_len=None, scales=None,
                       softmax_scale=None, out=None, return_lse=False, stream=None):
    """Attention of each query token over its own list of positions (what ``topk_indices`` returns).

    ``q`` and ``page_table`` as in ``tree_attention``.  ``indices``: int32 [batch, tokens, k]
    positions of sequence b, in any order, shared by the token's heads; negative entries are
    skipped, entries at or beyond ``kv_len[b]`` (int32 [batch], optional) are skipped and
    reported by ``device_status``.  Returns as ``tree_attention`` does.
    """
    c, dev = _cache(k_cache, v_cache, scales), k_cache.device
    batch, tokens = q.shape[0], q.shape[1]
    if indices.dim() != 3:
        raise ValueError("indices must be an int32 CUDA tensor [batch, tokens, k]")
    k = indices.shape[2]
    idx = _ints(indices, (batch, tokens, k), dev, "indices")
    limit = None if kv_len is None else _ints(kv_len, (batch,), dev, "kv_len")
    return _attend(q, c, dev, page_table, softmax_scale, out, return_lse, stream, "tks_selected_attention",
                   lambda cache, queries, handle: _lib().tks_selected_attention(cache, queries, idx, k, limit, handle))


def tree_mask(parents):
    """The bits ``tree_attention`` takes, from each draft's parent.

    ``parents``: an integer tensor [batch, tokens]; the parent of draft i is an earlier draft
    of the same sequence, or -1 for one that follows the context directly.  A draft attends to
    itself, its parent, its parent's parent and so on.  Returns int32 [batch, tokens,
    ceil(tokens / 32)] on the parents' device.
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


def _lib():
    from . import load
    return load()
