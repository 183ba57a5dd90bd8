"""The block and page entry points refuse bad arguments before any CUDA call."""

import ctypes

import pytest

import sparse_attention_topk_gb300 as tks
from tests.test_attention_abi import BAD_CACHES, cache, queries

OK_BOUNDS = dict(bounds=4096, block=8, pages=4, page_size=16, kv_heads=2, head_dim=64)


def bounds(**k):
    return ctypes.byref(tks.Bounds(**{**OK_BOUNDS, **k}))


BAD_BOUNDS = [dict(bounds=None), dict(bounds=4104), dict(block=0), dict(block=3), dict(block=32), dict(block=-8), dict(pages=0), dict(page_size=12),
              dict(page_size=0), dict(kv_heads=0), dict(head_dim=96), dict(pages=1 << 28)]
OTHER_BOUNDS = [dict(pages=5), dict(page_size=32), dict(kv_heads=1), dict(head_dim=128)]
INVAL = tks.TKS_E_INVAL


def call_bounds(c=None, b=None, table=64, stride=4, width=4, batch=1, start=None, end=64):
    return tks.load().tks_cache_bounds(c or cache(), b or bounds(), table, stride, width, batch, start, end, None)


def call_scores(b=None, q=None, kv_len=64, first=0, last=0, scores=64, n=8, row_len=64):
    return tks.load().tks_block_scores(b or bounds(), q or queries(out=None, softmax_scale=float("nan")), kv_len, first, last, scores, n, row_len, None)


def call_attention(c=None, q=None, blocks=64, n=2, block=8, kv_len=None):
    return tks.load().tks_block_attention(c or cache(), q or queries(), blocks, n, block, kv_len, None)


def call_fork(table=1 << 20, stride=4, width=4, sequences=2, lens=64, parents=64, new_lens=64, children=2, keep=None, pages=8, page=16, out=4096,
              src=64, dst=64, scratch=64):
    return tks.load().tks_cache_fork(table, stride, width, sequences, lens, parents, new_lens, children, keep, pages, page, out, src, dst, scratch, None)


def call_compact(table=1 << 20, stride=4, width=4, sequences=2, lens=64, keep=None, pages=8, page=16, out=4096, src=64, dst=64, count=64, scratch=64):
    return tks.load().tks_cache_compact(table, stride, width, sequences, lens, keep, pages, page, out, src, dst, count, scratch, None)


def call_copy(c=None, b=None, src=64, dst=64, n=2, count=None):
    return tks.load().tks_cache_copy(c or cache(), b, src, dst, n, count, None)


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(bad):
    c = cache(**bad)
    assert call_bounds(c) == call_attention(c) == call_copy(c) == INVAL


@pytest.mark.parametrize("bad", BAD_BOUNDS, ids=str)
def test_bad_bounds(bad):
    b = bounds(**bad)
    assert call_bounds(b=b) == call_scores(b) == call_copy(b=b) == INVAL


@pytest.mark.parametrize("other", OTHER_BOUNDS, ids=str)
def test_bounds_of_another_cache(other):
    assert call_bounds(b=bounds(**other)) == call_copy(b=bounds(**other)) == INVAL


@pytest.mark.parametrize("bad", [dict(table=None), dict(table=66), dict(stride=-4), dict(width=-1), dict(batch=-1), dict(start=66), dict(end=None),
                                 dict(end=66), dict(stride=1 << 57)], ids=str)
def test_bad_lengths_and_tables(bad):
    assert call_bounds(**bad) == INVAL


@pytest.mark.parametrize("bad", [dict(kv_len=66), dict(first=-1), dict(last=-1), dict(scores=None), dict(scores=66), dict(n=-1), dict(n=9), dict(row_len=66),
                                 dict(q=queries(q=None)), dict(q=queries(q_heads=7)), dict(q=queries(q_head_stride=4)), dict(q=queries(page_table=None)),
                                 dict(q=queries(batch=-1)), dict(q=queries(q=4098))], ids=str)
def test_bad_scores(bad):
    assert call_scores(**bad) == INVAL


@pytest.mark.parametrize("bad", [dict(blocks=None), dict(blocks=66), dict(n=-1), dict(block=0), dict(block=6), dict(block=-8), dict(kv_len=66),
                                 dict(n=tks.TKS_K_MAX, block=2), dict(n=1, block=1 << 25), dict(q=queries(out=None)),
                                 dict(q=queries(softmax_scale=float("inf")))], ids=str)
def test_bad_block_attention(bad):
    assert call_attention(**bad) == INVAL


@pytest.mark.parametrize("bad", [dict(table=None), dict(table=66), dict(stride=-1), dict(width=-1), dict(sequences=-1), dict(lens=None), dict(lens=66),
                                 dict(parents=None), dict(parents=66), dict(new_lens=None), dict(new_lens=66), dict(children=-1), dict(pages=0), dict(page=12),
                                 dict(page=0), dict(pages=1 << 30), dict(out=None), dict(out=66), dict(src=None), dict(dst=None), dict(scratch=None),
                                 dict(src=66), dict(dst=66), dict(scratch=68), dict(out=1 << 20), dict(out=(1 << 20) + 28), dict(out=(1 << 20) - 28)], ids=str)
def test_bad_forks(bad):
    assert call_fork(**bad) == INVAL


@pytest.mark.parametrize("bad", [dict(table=None), dict(table=66), dict(stride=-1), dict(width=-1), dict(sequences=-1), dict(lens=None), dict(lens=66),
                                 dict(pages=0), dict(page=12), dict(pages=1 << 30), dict(out=None), dict(out=66), dict(src=None), dict(dst=None),
                                 dict(count=None), dict(scratch=None), dict(count=66), dict(scratch=68), dict(out=(1 << 20) + 4),
                                 dict(out=1 << 20, stride=5)], ids=str)
def test_bad_compactions(bad):
    assert call_compact(**bad) == INVAL


@pytest.mark.parametrize("bad", [dict(src=None), dict(dst=None), dict(src=66), dict(dst=66), dict(n=-1), dict(count=66)], ids=str)
def test_bad_copies(bad):
    assert call_copy(**bad) == INVAL


def test_sizes_beyond_32_bits():
    assert call_fork(children=1 << 16, width=1 << 16, stride=1 << 16, sequences=1) == tks.TKS_E_TOO_LARGE
    assert call_compact(sequences=1 << 16, width=1 << 16, stride=1 << 16) == tks.TKS_E_TOO_LARGE


def test_nothing_to_do_is_no_error():
    assert call_bounds(batch=0, table=None, end=None) == tks.TKS_OK
    assert call_copy(n=0, src=None, dst=None) == tks.TKS_OK
    assert call_fork(children=0, parents=None, new_lens=None, src=None, dst=None, out=None, scratch=None) == tks.TKS_OK
    for none in (dict(batch=0), dict(tokens=0)):
        assert call_scores(q=queries(q=None, out=None, **none), scores=None, row_len=None) == tks.TKS_OK
        assert call_attention(q=queries(q=None, out=None, **none), blocks=None) == tks.TKS_OK


def test_no_device_is_reported_not_faked():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for rc in (call_bounds(), call_scores(), call_attention(), call_fork(), call_compact(), call_copy()):
        assert rc in (tks.TKS_E_UNSUPPORTED, tks.TKS_E_CUDA)


def test_status_string_of_a_full_pool():
    assert "free page" in tks.status_string(tks.TKS_E_NO_PAGE)


def test_cpu_tensors_are_refused():
    torch = pytest.importorskip("torch")
    i, c = torch.zeros(1, dtype=torch.int32), torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    t, b, q = i[None], torch.zeros(2, 2, 1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    for call in (lambda: tks.cache_bounds(c, t, i, b), lambda: tks.block_scores(q, b, t, t, 2), lambda: tks.block_attention(q, c, c, t, t[None, None], 2),
                 lambda: tks.cache_fork(t, i, i, i, 2, 4), lambda: tks.cache_compact(t, i, 2, 4), lambda: tks.cache_copy(i, i, c, c)):
        with pytest.raises(ValueError):
            call()
