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
