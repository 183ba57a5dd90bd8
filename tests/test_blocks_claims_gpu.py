"""What the block operators say of themselves beside their formulas."""

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.blocks_plain import bounds_of  # noqa: E402
from tests.test_blocks_gpu import HELD, check_bounds, filled, gen, ints, keys_of, new_bounds, sequence_bounds  # noqa: E402


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert tks.device_status() == tks.TKS_OK


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("tokens", [1, 20])
def test_by_how_much_a_product_exceeds_its_score(tokens, held):
    """Over bfloat16 by the sum's rounding alone (2 * 64 terms, each addition off by 2^-23 of their magnitudes at most); over 8 bits
    by half a step of the bounds, 2^-8, too. Queries of one sign in every channel make these add up."""
    lens = [500, 61]
    cache, table, _ = filled(lens, 32, 2, 64, held)
    bounds = new_bounds(cache, 16)
    tks.cache_bounds(cache.k, table, ints(lens), bounds, scales=cache.scales)
    for same_sign in (False, True):
        q = torch.randn(2, tokens, 8, 64, device="cuda", generator=gen(1)).to(torch.bfloat16)
        q = q.abs() if same_sign else q
        scores, seen = tks.block_scores(q, bounds, table, ints([[n] * tokens for n in lens]), 16)
        for b, n in enumerate(lens):
            k = keys_of(cache, table[b], n).double()
            for j in range(seen[b, 0, 0]):
                rows = k[16 * j : 16 * j + 16]
                for h in range(8):
                    x, size = q[b, :, h].double(), rows[:, h // 4].abs().amax(0)
                    most = (x @ rows[:, h // 4].T).amax(1)
                    room = (x.abs() @ size) * (129 * 2.0 ** -23 + (2.0 ** -8 if held == "int8" else 0.0))
                    assert (most <= scores[b, :, h // 4, j].double() + room).all()


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("layout", ["heads", "side by side"])
def test_bounds_of_other_layouts_leave_the_others(layout, held):
    lens = [77, 300]
    cache, table, _ = filled(lens, 32, 2, 128, held, layout)
    for starts in (None, [70, 130]):
        bounds = new_bounds(cache, 16, 3.0)
        before = bounds.clone()
        tks.cache_bounds(cache.k, table, ints(lens), bounds, start=None if starts is None else ints(starts), scales=cache.scales)
        check_bounds(cache, table, lens, starts or [0, 0], 16, bounds, before)


def test_bounds_of_lengths_that_are_held_to_the_table():
    cache, table, _ = filled([48, 40], 16, 1, 64, "int8", room=0)
    bounds = new_bounds(cache, 8, 5.0)
    before = bounds.clone()
    tks.cache_bounds(cache.k, table, ints([10 ** 6, -4]), bounds, start=ints([30, -9]), scales=cache.scales)
    assert tks.device_status() == tks.TKS_E_ROW_LEN
    want = bounds_of(keys_of(cache, table[0], 48), 8)
    got = sequence_bounds(bounds, table[0], 16, 6)
    assert torch.equal(got[3:].float(), want[3:].float()) and (got[:3] == 5.0).all()
    others = torch.ones(bounds.shape[0], dtype=torch.bool, device="cuda")
    others[table[0].long()] = False
    assert torch.equal(bounds[others], before[others])


@pytest.mark.parametrize("first, last", [(0, 0), (1, 1), (32, 0), (33, 31), (0, 65), (40, 2 ** 31 - 1)])
@pytest.mark.parametrize("lengths", ["equal", "causal", "none"])
def test_scores_of_chunks_are_the_same_where_none_is_forced(lengths, first, last):
    """(Whether scores take the short way is decided for 32 blocks at a time.)"""
    g, n, tokens = gen(6), 300, 90
    bounds = torch.randn(n, 1, 2, 2, 64, device="cuda", generator=g).sort(3).values.to(torch.bfloat16)
    table = torch.randperm(n, device="cuda", generator=g).to(torch.int32)[None]
    table[0, 270] = -1  # (reported where a token sees it)
    q = torch.randn(1, tokens, 8, 64, device="cuda", generator=g).to(torch.bfloat16)
    kv = {"equal": ints([[269 * 8] * tokens]), "causal": ints([[8 * 180 + t for t in range(tokens)]]), "none": ints([[0] * tokens])}[lengths]
    want, seen = tks.block_scores(q, bounds, table, kv, 8)
    got, again = tks.block_scores(q, bounds, table, kv, 8, first=first, last=last)
    j = torch.arange(n, device="cuda")
    forced = ((j < first) | (j >= seen.unsqueeze(-1).long() - last)) & (j < seen.unsqueeze(-1))
    assert torch.equal(seen, again) and torch.equal(got, torch.where(forced, math.inf, want))
