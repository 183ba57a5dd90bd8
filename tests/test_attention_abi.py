"""The cache and attention entry points refuse bad arguments before any CUDA call."""

import ctypes

import pytest

import sparse_attention_topk_gb300 as tks

OK_CACHE = dict(k=4096, v=8192, scales=64, held=tks.TKS_I8, pages=4, page_size=16, kv_heads=2, head_dim=64,
                page_stride=2048, token_stride=128, head_stride=64)
OK_Q = dict(q=4096, q_batch_stride=512, q_token_stride=512, q_head_stride=64, out=4096, lse=None, batch=1, tokens=1, q_heads=8,
            page_table=64, table_stride=4, table_pages=4, softmax_scale=0.125)


def cache(**k):
    return ctypes.byref(tks.Cache(**{**OK_CACHE, **k}))


def queries(**k):
    return ctypes.byref(tks.Queries(**{**OK_Q, **k}))


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=4104), dict(v=8200), dict(scales=None), dict(scales=68), dict(held=0), dict(held=3),
              dict(pages=0), dict(pages=-1), dict(page_size=0), dict(page_size=12), dict(pages=1 << 30), dict(kv_heads=0), dict(head_dim=96),
              dict(head_dim=0), dict(page_stride=-2048), dict(token_stride=120), dict(head_stride=1 << 62), dict(page_stride=1 << 60)]
BAD_QUERIES = [dict(q=None), dict(q=4098), dict(out=None), dict(out=4100), dict(lse=2), dict(batch=-1), dict(tokens=-1), dict(q_heads=7),
               dict(q_heads=0), dict(page_table=None), dict(page_table=66), dict(table_pages=-1), dict(table_stride=-1),
               dict(softmax_scale=float("inf")), dict(softmax_scale=float("nan")), dict(q_token_stride=-8), dict(q_head_stride=4),
               dict(batch=1 << 30, tokens=1 << 10), dict(q_batch_stride=1 << 62)]


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(bad):
    lib, c = tks.load(), cache(**bad)
    assert lib.tks_cache_write(c, 4096, 4096, 1, 1, 128, 64, 128, 64, 64, None) == tks.TKS_E_INVAL
    assert lib.tks_cache_read(c, 64, 1, 4096, 4096, 1, None) == tks.TKS_E_INVAL
    assert lib.tks_tree_attention(c, queries(), 64, None, None, None) == tks.TKS_E_INVAL
    assert lib.tks_selected_attention(c, queries(), 64, 8, None, None) == tks.TKS_E_INVAL


@pytest.mark.parametrize("bad", BAD_QUERIES, ids=str)
def test_bad_queries(bad):
    lib, q = tks.load(), queries(**bad)
    assert lib.tks_tree_attention(cache(), q, 64, None, None, None) == tks.TKS_E_INVAL
    assert lib.tks_selected_attention(cache(), q, 64, 8, None, None) == tks.TKS_E_INVAL


def test_null_structures():
    lib = tks.load()
    assert lib.tks_cache_write(None, 4096, 4096, 1, 1, 128, 64, 128, 64, 64, None) == tks.TKS_E_INVAL
    assert lib.tks_cache_read(None, 64, 1, 4096, 4096, 1, None) == tks.TKS_E_INVAL
    assert lib.tks_tree_attention(None, queries(), 64, None, None, None) == tks.TKS_E_INVAL
    assert lib.tks_tree_attention(cache(), None, 64, None, None, None) == tks.TKS_E_INVAL
    assert lib.tks_selected_attention(cache(), None, 64, 8, None, None) == tks.TKS_E_INVAL


@pytest.mark.parametrize("args", [
    # k, v, n, dtype, k strides, v strides, slots
    (None, 4096, 1, 1, 128, 64, 128, 64, 64), (4096, None, 1, 1, 128, 64, 128, 64, 64), (4096, 4096, -1, 1, 128, 64, 128, 64, 64),
    (4096, 4096, 1, 2, 128, 64, 128, 64, 64), (4096, 4096, 1, 1, 128, 64, 128, 64, None), (4096, 4096, 1, 1, 128, 64, 128, 64, 66),
    (4104, 4096, 1, 1, 128, 64, 128, 64, 64), (4096, 4096, 1, 1, -128, 64, 128, 64, 64), (4096, 4096, 1, 1, 128, 64, 128, 60, 64),
    (4096, 4096, 1, 0, 130, 64, 128, 64, 64), (4096, 4096, 1 << 30, 1, 128, 64, 128, 64, 64), (4096, 4096, 4, 1, 1 << 60, 64, 128, 64, 64)])
def test_bad_writes(args):
    assert tks.load().tks_cache_write(cache(), *args, None) == tks.TKS_E_INVAL


@pytest.mark.parametrize("args", [
    (None, 1, 4096, 4096, 1), (66, 1, 4096, 4096, 1), (64, -1, 4096, 4096, 1), (64, 1, None, 4096, 1), (64, 1, 4096, 4104, 1),
    (64, 1, 4096, 4096, 2), (64, 1 << 30, 4096, 4096, 1)])
def test_bad_reads(args):
    assert tks.load().tks_cache_read(cache(), *args, None) == tks.TKS_E_INVAL


def test_bad_lists_and_lengths():
    lib = tks.load()
    assert lib.tks_tree_attention(cache(), queries(), None, None, None, None) == tks.TKS_E_INVAL
    for args in ((66, None, None), (64, 66, None), (64, None, 66)):
        assert lib.tks_tree_attention(cache(), queries(), *args, None) == tks.TKS_E_INVAL
    assert lib.tks_tree_attention(cache(), queries(tokens=tks.TKS_DRAFTS_MAX + 1), 64, None, None, None) == tks.TKS_E_INVAL
    for args in ((None, 8, None), (66, 8, None), (64, -1, None), (64, tks.TKS_K_MAX + 1, None), (64, 8, 66)):
        assert lib.tks_selected_attention(cache(), queries(), *args, None) == tks.TKS_E_INVAL


def test_nothing_to_do_is_no_error():
    lib = tks.load()
    assert lib.tks_cache_write(cache(), None, None, 0, 1, 0, 0, 0, 0, None, None) == tks.TKS_OK
    assert lib.tks_cache_read(cache(), None, 0, None, None, 1, None) == tks.TKS_OK
    for none in (dict(batch=0), dict(tokens=0)):
        assert lib.tks_tree_attention(cache(), queries(q=None, out=None, **none), None, None, None, None) == tks.TKS_OK
        assert lib.tks_selected_attention(cache(), queries(q=None, out=None, **none), None, 8, None, None) == tks.TKS_OK


def test_no_device_is_reported_not_faked():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    lib = tks.load()
    for rc in (lib.tks_cache_write(cache(), 4096, 4096, 1, 1, 128, 64, 128, 64, 64, None), lib.tks_cache_read(cache(), 64, 1, 4096, 4096, 1, None),
               lib.tks_tree_attention(cache(), queries(), 64, None, None, None), lib.tks_selected_attention(cache(), queries(), 64, 8, None, None)):
        assert rc in (tks.TKS_E_UNSUPPORTED, tks.TKS_E_CUDA)


def test_status_string_of_a_bad_index():
    assert "outside the cache" in tks.status_string(tks.TKS_E_INDEX)


def test_cpu_tensors_are_refused():
    torch = pytest.importorskip("torch")
    c = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tks.cache_read(c, c, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        tks.tree_attention(torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16), c, c, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_tree_mask():
    torch = pytest.importorskip("torch")
    #   0   1      two roots; 2 and 3 below 0, 4 below 3
    bits = tks.tree_mask(torch.tensor([[-1, -1, 0, 0, 3]]))
    assert bits.tolist() == [[[0b1], [0b10], [0b101], [0b1001], [0b11001]]] and bits.dtype is torch.int32
    chain = tks.tree_mask(torch.arange(-1, 39)[None])
    assert chain[0, 39].tolist() == [-1, 0xFF] and chain[0, 31].tolist() == [-1, 0] and chain[0, 30].tolist() == [0x7FFFFFFF, 0]
    assert tks.tree_mask(torch.zeros(2, 0, dtype=torch.int64)).shape == (2, 0, 0)
    with pytest.raises(ValueError):
        tks.tree_mask(torch.tensor([[-1, 1]]))
    with pytest.raises(ValueError):
        tks.tree_mask(torch.tensor([[-2]]))
