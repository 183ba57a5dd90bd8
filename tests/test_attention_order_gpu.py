"""Calls whose blocks have no work, one segment or several: what a warp's lanes and a cluster's
blocks leave for each other in shared memory has to be there when it is read, in every run."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.test_attention_gpu import HELD, selected_case, tree_case  # noqa: E402


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert tks.device_status() == tks.TKS_OK


def same_bits(case, times=8):
    out, lse = case()
    for _ in range(times):
        o, l = case()
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads", [8, 80])
@pytest.mark.parametrize("ctx", [[5], [0, 70], [1, 0, 300, 64]])
def test_clusters_of_which_some_blocks_have_no_work(ctx, q_heads, held):
    """Page tables that could hold 1600 positions more than the sequences have."""
    same_bits(lambda: tree_case(ctx, 1, q_heads, 2, 64, held, 16, room=100))


@pytest.mark.parametrize("held", HELD)
def test_blocks_of_several_segments(held):
    """More units than blocks, 32 rows of each, and lists of one to three tiles."""
    same_bits(lambda: tree_case([(61 * i) % 300 for i in range(60)], 4, 64, 8, 64, held, 16), 4)
    selected_case([300], 500, 70, 64, 1, 64, held, 16)
