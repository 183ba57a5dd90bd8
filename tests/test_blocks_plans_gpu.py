"""Block attention in whole units (lists that thread blocks take one after the other, without the joining kernel) and in equal runs,
on both sides of the rule that chooses; scores that are more than stay in L2."""

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.attention_plain import check_rows  # noqa: E402
from tests.test_blocks_gpu import HELD, filled, gen, ints  # noqa: E402


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert tks.device_status() == tks.TKS_OK


def attend(seen, tokens, q_heads, kv_heads, dim, held, page, block, chosen, width=None, seed=0):
    """Every token and head against the definition: keys of ragged lists, some empty, some with -1 among the blocks."""
    g = gen(seed)
    lens = [max(x) for x in seen]
    cache, table, rows = filled(lens, page, kv_heads, dim, held, seed=seed)
    if width is not None:
        table = torch.nn.functional.pad(table, (0, width - table.shape[1]), value=-1)
    q = (1.5 * torch.randn(len(seen), tokens, q_heads, dim, device="cuda", generator=g)).to(torch.bfloat16)
    kv = ints(seen)
    blocks = (kv + block - 1) // block
    # a random order of each token's blocks, cut to a length of its own
    most = int(blocks.max())
    order = torch.rand(len(seen), tokens, kv_heads, most, device="cuda", generator=g)
    order.masked_fill_(torch.arange(most, device="cuda") >= blocks[..., None, None], 2.0)
    value, lists = order.sort(-1)
    lists = torch.nn.functional.pad(torch.where(value < 2.0, lists, -1), (0, max(0, chosen - most)), value=-1)[..., :chosen]
    cut = torch.randint(0, 2 * chosen, (len(seen), tokens, kv_heads, 1), device="cuda", generator=g)  # (half of them stay whole)
    lists = torch.where(torch.arange(chosen, device="cuda") < cut, lists, -1).to(torch.int32)
    lists = lists.gather(-1, torch.rand(lists.shape, device="cuda", generator=g).argsort(-1))
    out, lse = tks.block_attention(q, cache.k, cache.v, table, lists, block, kv_len=kv, scales=cache.scales, return_lse=True)
    group = q_heads // kv_heads
    host = lists.tolist()
    for b in range(len(seen)):
        for t in range(tokens):
            for h in range(kv_heads):
                pos = [x * block + i for x in host[b][t][h] if x >= 0 for i in range(block) if x * block + i < seen[b][t]]
                pos = torch.tensor(pos, dtype=torch.long, device="cuda")
                hs = slice(h * group, (h + 1) * group)
                check_rows(out[b, t, hs], lse[b, t, hs], q[b, t, hs].double(), rows[b][0][pos, h], rows[b][1][pos, h],
                           torch.ones(group, len(pos), dtype=torch.bool, device="cuda"), dim ** -0.5, held)
    again = tks.block_attention(q, cache.k, cache.v, table, lists, block, kv_len=kv, scales=cache.scales, return_lse=True)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def ragged(sequences, tokens, most):
    return [[(most * 7 // 10 + 131 * (b * tokens + t)) % most + (t > 0) for t in range(tokens)] for b in range(sequences)]


# Lists: 304 places of two thread blocks an SM; whole units where ceil(units / 304) * 304 - units empty ones times (5 + tiles of a
# list) are at most 12 * 304.
@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("sequences, tokens, chosen", [(1, 151, 6), (1, 152, 6), (8, 19, 6), (1, 153, 6), (3, 101, 6), (4, 76, 4), (2, 152, 9), (2, 200, 12)])
def test_lists_about_as_many_as_places(sequences, tokens, chosen, held):
    """Of 2 heads: 302, 304, 304, 306 (nearly all of a second round empty: equal runs), 606, 608, 608 and 800 units."""
    attend(ragged(sequences, tokens, 700), tokens, 8, 2, 128, held, 32, 32, chosen, width=400)


# bfloat16 lists that are together longer than the sequence: 456 places of three thread blocks an SM.
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens, chosen", [(227, 8), (228, 8), (229, 8), (455, 5), (456, 5)])
def test_bfloat16_lists_out_of_l2_about_as_many_as_places(tokens, chosen, dim):
    attend(ragged(1, tokens, 600), tokens, 6, 2, dim, "bf16", 64, 32, chosen)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("page, block", [(8, 16), (64, 4), (16, 1)])
def test_whole_lists_looked_up_by_the_key(page, block, held):
    attend(ragged(2, 152, 400), 152, 4, 1, 64, held, page, block, 192 // block)


@pytest.mark.parametrize("tokens, q_heads, kv_heads, first, last", [(2100, 4, 1, 0, 0), (2100, 4, 1, 1, 1), (1050, 6, 2, 0, 0), (70, 129, 1, 2, 0)])
def test_scores_that_do_not_stay_in_l2(tokens, q_heads, kv_heads, first, last):
    """More than 2^24 of them."""
    g = gen(4)
    n = 2 ** 24 // (tokens * kv_heads) + 9
    bounds = torch.randn(300, 4, kv_heads, 2, 64, device="cuda", generator=g).sort(3).values.to(torch.bfloat16)
    table = torch.randint(300, (1, n // 4 + 1), device="cuda", generator=g).to(torch.int32)
    q = torch.randn(1, tokens, q_heads, 64, device="cuda", generator=g).to(torch.bfloat16)
    kv = (torch.randint(1, n + 1, (1, tokens), device="cuda", generator=g) * 16).to(torch.int32)
    kv[:, ::3] = 16 * n
    kv[0, 5] = 0
    scores, seen = tks.block_scores(q, bounds, table, kv, 16, first=first, last=last, n=n)
    assert scores.numel() > 2 ** 24 and torch.equal(seen, (kv // 16).unsqueeze(-1).expand(-1, -1, kv_heads))
    j = torch.arange(n, device="cuda")
    mine = bounds[table[0, j // 4].long(), j % 4]
    group = q_heads // kv_heads
    step = max(1, 2 ** 22 // (n * group))
    for h in range(kv_heads):
        lo, hi = mine[:, h, 0].double(), mine[:, h, 1].double()
        most = torch.maximum(lo.abs(), hi.abs())
        for t in range(0, tokens, step):
            x = q[0, t : t + step, h * group : (h + 1) * group].double()
            want = (x.clamp(min=0) @ hi.T + x.clamp(max=0) @ lo.T).amax(1)
            room = (x.abs() @ most.T).amax(1) * 128 * 2.0 ** -23
            there = seen[0, t : t + step, h, None]
            want = torch.where((j < first) | (j >= there - last), math.inf, want)
            want = torch.where(j >= there, -math.inf, want)
            got = scores[0, t : t + step, h].double()
            ok = (got == want) | ((got - want).abs() <= room)
            assert ok.all()
