"""Chains of drafted tokens without a mask, up to a chunk of a prompt."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.test_attention_gpu import HELD, tree_case  # noqa: E402


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert tks.device_status() == tks.TKS_OK


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("drafts, q_heads, kv_heads", [(16, 1, 1), (31, 2, 2), (65, 8, 2), (257, 4, 1), (1024, 2, 1)])
def test_chains(drafts, q_heads, kv_heads, held):
    tree_case([0, 333], drafts, q_heads, kv_heads, 64, held, 16, tree=None, counts=[drafts, max(1, drafts - 3)], seed=drafts)
    tree_case([1000], drafts, q_heads, kv_heads, 128, held, 64, tree=None, seed=drafts)
