"""A scale that is finite but leaves 32 bits as a power of two is refused, before any CUDA call."""

import pytest

import sparse_attention_topk_gb300 as tks
from tests.test_attention_abi import cache, queries


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.4e38])
def test_scales_beyond_the_range(scale):
    lib = tks.load()
    assert lib.tks_tree_attention(cache(), queries(softmax_scale=scale), 64, None, None, None) == tks.TKS_E_INVAL
    assert lib.tks_selected_attention(cache(), queries(softmax_scale=scale), 64, 8, None, None) == tks.TKS_E_INVAL


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.3e38, 2.4e38])
def test_the_largest_scale(scale):
    """Queries of zeros: every score is 0 and the result the values' mean, or the call is refused."""
    torch = pytest.importorskip("torch")
    for heads in (1, 40):
        q = torch.zeros(1, 1, heads, 64, dtype=torch.bfloat16, device="cuda")
        k, v = (torch.ones(2, 16, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        table, ctx = torch.arange(2, dtype=torch.int32, device="cuda")[None], torch.tensor([30], dtype=torch.int32, device="cuda")
        if scale > 2.3e38:
            with pytest.raises(ValueError):
                tks.tree_attention(q, k, v, table, ctx, softmax_scale=scale)
        else:
            assert (tks.tree_attention(q, k, v, table, ctx, softmax_scale=scale) == 1).all()
    assert tks.device_status() == tks.TKS_OK
