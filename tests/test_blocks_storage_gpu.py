"""What the tensors that block and page calls return hold on to."""

import io

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def saved(x):
    f = io.BytesIO()
    torch.save(x, f)
    size = f.tell()
    f.seek(0)
    return torch.load(f), size


@pytest.mark.parametrize("columns", [1, 40, 3000])
def test_scores_and_row_lengths_are_saved_together(columns):
    bounds = torch.randn(30, 2, 2, 2, 64, device="cuda").to(torch.bfloat16)
    q = torch.randn(3, 50, 4, 64, device="cuda").to(torch.bfloat16)
    table = torch.randint(30, (3, (columns + 1) // 2), device="cuda").to(torch.int32)
    scores, seen = tks.block_scores(q, bounds, table, None, 8, n=columns)
    (a, b), _ = saved((scores, seen))
    assert torch.equal(a, scores) and torch.equal(b, seen)
    assert scores.untyped_storage().data_ptr() != seen.untyped_storage().data_ptr()
    assert scores.untyped_storage().nbytes() == 4 * scores.numel() and seen.untyped_storage().nbytes() == 4 * seen.numel()
    assert tks.device_status() == tks.TKS_OK


def owns(*tensors):
    assert len({t.untyped_storage().data_ptr() for t in tensors}) == len(tensors)
    for t in tensors:
        assert t.untyped_storage().nbytes() == 4 * t.numel()
        a, size = saved(t)
        assert torch.equal(a, t) and size < 4 * t.numel() + 4096


@pytest.mark.parametrize("children", [2, 100])
@pytest.mark.parametrize("pages", [64, 9000, 400_000])
def test_what_a_fork_returns_holds_nothing_else(pages, children):
    table, lens = ints([[5, 7, -1]]), ints([20])
    owns(*tks.cache_fork(table, lens, ints([0] * children), ints([20] * children), pages, 16))
    assert tks.device_status() == tks.TKS_OK


@pytest.mark.parametrize("pages", [64, 9000, 400_000])
def test_what_a_compaction_returns_holds_nothing_else(pages):
    owns(*tks.cache_compact(ints([[5, 7, -1]]), ints([20]), pages, 16))
    assert tks.device_status() == tks.TKS_OK


def test_a_pool_of_one_page_has_no_moves():
    table, src, dst, count = tks.cache_compact(ints([[0, -1]]), ints([3]), 1, 4)
    assert table.tolist() == [[0, -1]] and src.numel() == dst.numel() == 0 and count.tolist() == [0, 1]
    assert tks.device_status() == tks.TKS_OK
